// Low-rank adapters of many requests beside a packed projection.
//
//   t[m][j] = s_a sum_k x[m][k] A[a][j][k]            a = ids[m], the adapter of row m
//   y[m][n] = sum_k x[m][k] W[n][k] + sum_j t[m][j] B[a][n][j]
//
// A is bf16 [L][r][K], B bf16 [L][N][r], s fp32 [L]; a row with a negative id has no adapter.
//
// The first product ("shrink") reads every activation once more and the adapters in use; it is bound by that
// traffic, so it runs on mma.sync straight from global memory (ql_lora_dot.cuh): on the fused path in the kernel below,
// which converts the activations on the way, on the weight-streaming path in that kernel's idle warps.  The second
// ("expand") never makes a pass over y of its own: the weight-streaming path adds it in fp32 where it sums its partials
// (lora_reduce_kernel), the fused path appends it to the tile's K loop (ql_tc_fused.cuh), so y is rounded once.
#pragma once

#include "ql_lora_dot.cuh"
#include "ql_prepass.cuh"
#include "ql_ptx.cuh"
#include "ql_tc_fused.cuh"
#include "ql_tc_skinny.cuh"

namespace ql {
namespace lora {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSplit = 8;           // CTAs of a cluster that share a tile's K range

struct ShrinkParams {
    const __nv_bfloat16* x;      // [M][K]
    const __nv_bfloat16* a[2];   // [L][r][K]; the second one of a gate/up pair
    const float* scale;          // [L] or null (1)
    const int* ids;              // [M]
    int M, K, r, L;
    int tiles;                   // ceil(M / 32)
    int passes;                  // CTAs that share a tile's distinct adapters
    int chunks;                  // CTAs along the rank: ceil(r / (8 NT))
    __nv_bfloat16* tw;           // [M][pairs][r / 8][hi 8 | lo 8]: t 2^-e_m in two bf16 parts
    __half* xh;                  // [M][K]: x 2^-e_m in the dequantizer's k order
    float* rowscale;             // [M]: 2^e_m
    int bits, pairs;
    int* row_slot;               // [M] position of the row's adapter in its token tile's list, or -1
    int* tile_count;             // [num_t] distinct adapters of the token tile
    int* tile_list;              // [num_t][BT] those adapters, in order of first use
    int num_t;
};

// One token tile of the fused kernel: its distinct adapters in order of first use, and each row's place among them.
__device__ __forceinline__ void plan_tile(const ShrinkParams& p, int t_blk) {
    constexpr int BT = fused::BT;
    static_assert(BT <= kThreads, "one thread per token of a tile");
    __shared__ int id[BT];
    __shared__ int warp_first[kWarps];
    const int i = threadIdx.x;
    const int m = t_blk * BT + i;
    const int rows = min(BT, p.M - t_blk * BT);
    const int mine = i < rows ? adapter_of(p.ids, m, p.L) : -1;
    if (i < BT) id[i] = mine;
    __syncthreads();
    int first = i;                                 // the tile's first row with this adapter
    if (mine >= 0)
        for (int j = 0; j < i; ++j)
            if (id[j] == mine) { first = j; break; }
    const bool leads = mine >= 0 && first == i;
    const uint32_t bal = __ballot_sync(0xFFFFFFFFu, leads);
    if ((i & 31) == 0) warp_first[i >> 5] = __popc(bal);
    __syncthreads();
    int place = __popc(bal & ((1u << (i & 31)) - 1u)), total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < (i >> 5)) place += warp_first[w];
        total += warp_first[w];
    }
    __syncthreads();
    if (leads) {
        p.tile_list[t_blk * BT + place] = mine;
        id[i] = place;                             // only this row's entry: others read id[first] below
    }
    __syncthreads();
    if (i < rows) p.row_slot[m] = mine >= 0 ? id[first] : -1;
    if (i == 0) p.tile_count[t_blk] = total;
}

// The conversion's row scale (convert_x_kernel): 2^e with the row's largest magnitude in [2^15, 2^16) after division,
// 1 for a zero or non-finite row.  amax: the largest bf16 bit pattern without its sign.
__device__ __forceinline__ float row_scale(uint32_t amax) {
    const uint32_t ex = amax >> 7;                 // biased exponent
    if (amax == 0 || ex == 0xFF) return 1.0f;
    const int e = max(static_cast<int>(ex) - 127, -100) - 15;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The first product and the conversion for tiles of 32 rows.  grid: (tiles * passes + num_t, S, chunks * pairs),
// cluster (1, S, 1).
//
// Each warp multiplies its share of the K range, 32 columns at a time (dot_block).  The warps' sums meet in shared
// memory, the cluster's CTAs' in distributed shared memory, each added in a fixed order.
//
// Rows of a tile with other adapters are multiplied too and not written: a tile makes one pass per distinct adapter,
// and its passes are spread over `passes` CTAs.
//
// The same kernel converts the activations (as convert_x_kernel), whose row scale the extra K-steps share, so x comes
// from DRAM once: the maxima are taken from the registers that feed the MMAs, and the first pass's CTAs then read their
// rows again, from L2, to convert them.
template <int NT>
__global__ void __launch_bounds__(kThreads, 2) lora_shrink_kernel(const ShrinkParams p) {
    ptx::launch_dependents();
    constexpr int MT = 2, kRows = kTile * MT;
    constexpr int kSums = kRows * NT * 8;
    __shared__ float part[kWarps][kSums];          // [row][rank] per warp
    __shared__ uint32_t amax[kWarps][kRows];
    __shared__ float scale_s[kRows];
    const int S = static_cast<int>(gridDim.y);
    const int rank = static_cast<int>(blockIdx.y);             // rank in the cluster (1, S, 1)
    const int shrink_ctas = p.tiles * p.passes;
    if (static_cast<int>(blockIdx.x) >= shrink_ctas) {
        if (blockIdx.y == 0 && blockIdx.z == 0) plan_tile(p, static_cast<int>(blockIdx.x) - shrink_ctas);
    } else {
        const int tile = static_cast<int>(blockIdx.x) / p.passes, pass = static_cast<int>(blockIdx.x) % p.passes;
        const int pair = static_cast<int>(blockIdx.z) / p.chunks, chunk = static_cast<int>(blockIdx.z) % p.chunks;
        const bool converts = pass == 0 && blockIdx.z == 0;
        const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
        const int m0 = tile * kRows;
        const int j0 = chunk * NT * 8;
        const int mine = lane < kRows && m0 + lane < p.M ? adapter_of(p.ids, m0 + lane, p.L) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, mine);
        uint32_t leaders = __ballot_sync(0xFFFFFFFFu, mine >= 0 && (__ffs(same) - 1) == lane);
        const int kb_all = p.K / 32;
        const int kb0 = static_cast<int>(static_cast<int64_t>(kb_all) * rank / S);
        const int kb1 = static_cast<int>(static_cast<int64_t>(kb_all) * (rank + 1) / S);
        const int g = lane >> 2, c = lane & 3;
        const uint4* xr[2 * MT];
#pragma unroll
        for (int q = 0; q < 2 * MT; ++q) {         // rows past M repeat the last one; their results are not written
            const int64_t row = min(m0 + g + 8 * q, p.M - 1);
            xr[q] = reinterpret_cast<const uint4*>(p.x + row * p.K) + c;
        }
        bool first = true;                         // the pass that also takes the rows' maxima
        for (int n = 0; leaders != 0 || (converts && first); ++n, leaders &= leaders - 1) {
            if (leaders != 0 && n % p.passes != pass) continue;
            const bool with = leaders != 0;        // false: a converting CTA without an adapter in its rows
            const int adapter = with ? __shfl_sync(0xFFFFFFFFu, mine, __ffs(leaders) - 1) : -1;
            const __nv_bfloat16* a = (pair == 0 ? p.a[0] : p.a[1]) + (static_cast<int64_t>(with ? adapter : 0) * p.r + j0) * p.K;
            const int nt_live = with ? min(NT, p.r / 8 - chunk * NT) : 0;
            float acc[MT][NT][4];
#pragma unroll
            for (int q = 0; q < MT; ++q)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[q][i][e] = 0.0f;
            uint32_t mx[2 * MT];
#pragma unroll
            for (int q = 0; q < 2 * MT; ++q) mx[q] = 0u;
            constexpr int U = NT == 1 ? 4 : 2;                 // column blocks in flight per warp
            for (int kb = kb0 + warp; kb < kb1; kb += kWarps * U) {
                uint4 vx[U][2 * MT], va[U][NT];
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int b = kb + u * kWarps;
                    const bool in = b < kb1;
#pragma unroll
                    for (int q = 0; q < 2 * MT; ++q) vx[u][q] = in ? __ldg(xr[q] + 4 * b) : zero;
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        va[u][i] = in && i < nt_live
                                       ? __ldg(reinterpret_cast<const uint4*>(a + static_cast<int64_t>(8 * i + g) * p.K) + c + 4 * b)
                                       : zero;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (first) {
#pragma unroll
                        for (int q = 0; q < 2 * MT; ++q) {
                            const uint4 v = vx[u][q];
                            mx[q] = __vmaxu2(mx[q], __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                                             __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int q = 0; q < MT; ++q) dot_block(acc[q][i], vx[u][2 * q], vx[u][2 * q + 1], va[u][i]);
                }
            }
#pragma unroll
            for (int q = 0; q < MT; ++q)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int at = (16 * q + g) * NT * 8 + 8 * i + 2 * c;
                    *reinterpret_cast<float2*>(&part[warp][at]) = make_float2(acc[q][i][0], acc[q][i][1]);
                    *reinterpret_cast<float2*>(&part[warp][at + 8 * NT * 8]) = make_float2(acc[q][i][2], acc[q][i][3]);
                }
            if (first) {
#pragma unroll
                for (int q = 0; q < 2 * MT; ++q) {
                    uint32_t v = max(mx[q] & 0xFFFFu, mx[q] >> 16);
                    v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                    v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
                    if (c == 0) amax[warp][g + 8 * q] = v;
                }
            }
            __syncthreads();
            for (int e = threadIdx.x; e < kSums; e += kThreads) {
                float s = part[0][e];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) s += part[w][e];
                part[0][e] = s;                                // this CTA's slice of the sum
            }
            if (first && threadIdx.x < kRows) {
                uint32_t v = amax[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) v = max(v, amax[w][threadIdx.x]);
                amax[0][threadIdx.x] = v;
            }
            if (S > 1) ptx::cluster_sync(); else __syncthreads();
            if (first) {
                if (threadIdx.x < kRows) {
                    uint32_t v = amax[0][threadIdx.x];
                    for (int q = 0; S > 1 && q < S; ++q)
                        v = max(v, __float_as_uint(ptx::ld_shared_cluster_f32(&amax[0][threadIdx.x], static_cast<uint32_t>(q))));
                    const float sc = row_scale(v);
                    scale_s[threadIdx.x] = sc;
                    if (converts && rank == 0 && m0 + static_cast<int>(threadIdx.x) < p.M) p.rowscale[m0 + threadIdx.x] = sc;
                }
                __syncthreads();
            }
            // every CTA of the cluster finishes its share of the tile's sums, two ranks at a time
            for (int e = 2 * (static_cast<int>(threadIdx.x) + rank * kThreads); with && e < kSums; e += 2 * S * kThreads) {
                float s0 = part[0][e], s1 = part[0][e + 1];
                if (S > 1) {
                    s0 = s1 = 0.0f;
                    for (int q = 0; q < S; ++q) {
                        s0 += ptx::ld_shared_cluster_f32(&part[0][e], static_cast<uint32_t>(q));
                        s1 += ptx::ld_shared_cluster_f32(&part[0][e + 1], static_cast<uint32_t>(q));
                    }
                }
                const int row = e / (NT * 8), j = j0 + e % (NT * 8);
                const int m = m0 + row;
                if (m < p.M && j < p.r && p.ids[m] == adapter) {
                    const float sc = p.scale != nullptr ? __ldg(p.scale + adapter) : 1.0f;
                    s0 *= sc;
                    s1 *= sc;
                    const float inv = __uint_as_float(0x7F000000u - __float_as_uint(scale_s[row]));       // 2^-e_m
                    __nv_bfloat16* o = p.tw + (static_cast<int64_t>(m) * p.pairs + pair) * 2 * p.r + 16 * (j / 8) + j % 8;
                    *reinterpret_cast<uint32_t*>(o) = fused::bf16_part(s0 * inv, s1 * inv, false);
                    *reinterpret_cast<uint32_t*>(o + 8) = fused::bf16_part(s0 * inv, s1 * inv, true);
                }
            }
            if (S > 1) ptx::cluster_sync(); else __syncthreads();      // the sums are read before the next pass
            first = false;
            if (!with) break;
        }
        if (converts) {
            if (rank == 0) {
                // rows without an adapter: zeros in tw, so that a tile's box of it needs no mask
                const int pieces = p.pairs * p.r / 4;
                for (int row = warp; row < kRows && m0 + row < p.M; row += kWarps) {
                    if (__shfl_sync(0xFFFFFFFFu, mine, row) >= 0) continue;
                    uint4* o = reinterpret_cast<uint4*>(p.tw) + static_cast<int64_t>(m0 + row) * pieces;
                    for (int i = lane; i < pieces; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            // the CTA's columns of its rows, a row per warp at a time
            const int c0 = 4 * kb0, c1 = 4 * kb1;
            for (int row = warp; row < kRows && m0 + row < p.M; row += kWarps) {
                const float inv = __uint_as_float(0x7F000000u - __float_as_uint(scale_s[row]));
                const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(m0 + row) * p.K);
                uint4* dst = reinterpret_cast<uint4*>(p.xh + static_cast<int64_t>(m0 + row) * p.K);
                for (int i = c0 + lane; i < c1; i += 32 * 4) {
                    uint4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (i + 32 * u < c1) v[u] = __ldg(src + i + 32 * u);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (i + 32 * u < c1) dst[i + 32 * u] = p.bits == 4 ? convert8<4>(v[u], inv) : convert8<8>(v[u], inv);
                }
            }
        }
    }
    // Launched behind the parameter transpose under programmatic dependent launch; as with the conversion of the
    // plain layer, the last CTA waits for it, so that this kernel's completion implies both.
    if (blockIdx.x == gridDim.x - 1) ptx::grid_dependency_wait();
}

// y[t][n] = 2^rowexp[t] * (sum of the stream-K partials, as skinny_reduce_kernel) + sum_j t[t][j] B[a][n][j] with
// t = s sum_z tp[z], all in fp32 from the bf16 adapter, rounded once.  One CTA per (128-column tile, 2 tokens); a
// thread's first kEager chunks of B are loaded before the wait for the partials.
struct ExpandParams {
    const __nv_bfloat16* b;      // [L][N][r]
    const float* scale;          // [L] or null (1)
    const float* tp;             // [slices][M][r]
    const int* ids;              // [M]
    int r, L, slices;
};

template <bool kBf16Out>
__global__ void __launch_bounds__(256) lora_reduce_kernel(const float* __restrict__ partial,
                                                          const int* __restrict__ rowexp, void* __restrict__ y, int M,
                                                          int N, int cpt, int64_t units, int P, int segmax,
                                                          int64_t partial_elems, const ExpandParams ep) {
    __shared__ int64_t seg_base[skinny::kMaxCtas];
    __shared__ int count;
    __shared__ float ps[2][128];
    __shared__ __align__(16) float tl[2][kMaxRank];
    constexpr int kEager = 4;
    const int w = blockIdx.x;
    const int t = blockIdx.y * 2 + (threadIdx.x >> 7), n = w * skinny::BW + (threadIdx.x & 127);
    const bool live = t < M && n < N;
    if (threadIdx.x == 0) count = skinny::list_segments(w, cpt, units, P, segmax, seg_base);
    const int a = t < M ? ep.ids[t] : -1;
    const bool with = a >= 0 && a < ep.L;                         // the first product records an id out of range
    const int chunks = with && live ? ep.r / 8 : 0;
    const uint4* b = reinterpret_cast<const uint4*>(ep.b + (static_cast<int64_t>(with ? a : 0) * N + (live ? n : 0)) * ep.r);
    uint4 eager[kEager];
#pragma unroll
    for (int i = 0; i < kEager; ++i) eager[i] = i < chunks ? __ldg(b + i) : make_uint4(0u, 0u, 0u, 0u);
    const float sc = with && ep.scale != nullptr ? __ldg(ep.scale + a) : 1.0f;
    __syncthreads();
    ptx::grid_dependency_wait();                                  // partials and tp come from the kernel before
    // t of the CTA's two tokens: a token's 128 threads share out the slices, then add their sums in order
    const int half = threadIdx.x >> 7, i128 = threadIdx.x & 127;
    const int groups = 128 / ep.r, j = i128 % ep.r, group = i128 / ep.r;
    if (with && group < groups) {
        const float* tp = ep.tp + static_cast<int64_t>(t) * ep.r + j;
        const int64_t step = static_cast<int64_t>(M) * ep.r;
        float sum = 0.0f;
#pragma unroll 8
        for (int z = group; z < ep.slices; z += groups) sum += tp[z * step];
        ps[half][i128] = sum;
    }
    float acc = live ? skinny::sum_segments(partial, partial_elems, seg_base, count, M, t, i128) : 0.0f;
    __syncthreads();
    if (with && i128 < ep.r) {
        float sum = ps[half][i128];
        for (int q = 1; q < groups; ++q) sum += ps[half][i128 + q * ep.r];
        tl[half][i128] = sc * sum;
    }
    __syncthreads();
    if (!live) return;
    acc = ldexpf(acc, rowexp[t]);
    const float4* tt = reinterpret_cast<const float4*>(tl[half]);
    float delta = 0.0f;
    auto add = [&](const uint4 v, int i) {
        const float4 t0 = tt[2 * i], t1 = tt[2 * i + 1];
        const uint32_t q[4] = {finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w)};
        delta = fmaf(t0.x, bf16_lo(q[0]), delta);
        delta = fmaf(t0.y, bf16_hi(q[0]), delta);
        delta = fmaf(t0.z, bf16_lo(q[1]), delta);
        delta = fmaf(t0.w, bf16_hi(q[1]), delta);
        delta = fmaf(t1.x, bf16_lo(q[2]), delta);
        delta = fmaf(t1.y, bf16_hi(q[2]), delta);
        delta = fmaf(t1.z, bf16_lo(q[3]), delta);
        delta = fmaf(t1.w, bf16_hi(q[3]), delta);
    };
#pragma unroll
    for (int i = 0; i < kEager; ++i)
        if (i < chunks) add(eager[i], i);
    for (int i = kEager; i < chunks; ++i) add(__ldg(b + i), i);
    acc += delta;
    const int64_t e = static_cast<int64_t>(t) * N + n;
    if constexpr (kBf16Out) {
        reinterpret_cast<__nv_bfloat16*>(y)[e] = __float2bfloat16_rn(acc);
    } else {
        reinterpret_cast<float*>(y)[e] = acc;
    }
}

}  // namespace lora
}  // namespace ql
