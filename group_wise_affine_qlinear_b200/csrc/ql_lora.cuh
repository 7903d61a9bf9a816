// Low-rank adapters of many requests beside a packed projection.
//
//   t[m][j] = s_a sum_k x[m][k] A[a][j][k]            a = ids[m], the adapter of row m
//   y[m][n] = sum_k x[m][k] W[n][k] + sum_j t[m][j] B[a][n][j]
//
// A is bf16 [L][r][K], B bf16 [L][N][r], s fp32 [L]; a row with a negative id has no adapter.
//
// The first product ("shrink") reads every activation once more and the adapters in use: a flop per byte and rank, too
// few for the tensor core's large tiles, so it runs on mma.sync: on the fused path in the kernel below, fed by TMA, which
// converts the activations beside it, on the weight-streaming path straight from global memory in that kernel's drain
// warps (ql_lora_dot.cuh).  The second
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

constexpr int kThreads = 128;          // of the first product
constexpr int kWarps = kThreads / 32;
constexpr int kConvGroups = 4;         // pairs of warps that convert a row each
constexpr int kConvThreads = 64;       // of one such pair
constexpr int kBlock = kThreads + kConvGroups * kConvThreads;
constexpr int kRows = 2 * kTile;       // rows of one tile of the first product on the fused path
constexpr int kCols = 64;              // columns of one ring slot: 128-byte rows
constexpr int kSlots = 3;              // ring slots per warp
constexpr int kMaxSplit = 8;           // CTAs of a cluster that share a tile's K range
constexpr uint32_t kXSlot = kRows * kCols * 2;

// A ring slot: the tile's rows of x and 8 NT ranks of A, 64 columns each.
__host__ __device__ constexpr uint32_t slot_bytes(int nt) { return kXSlot + static_cast<uint32_t>(nt) * 8 * kCols * 2; }
__host__ __device__ constexpr uint32_t shrink_smem(int nt) { return kWarps * kSlots * slot_bytes(nt) + 1024; }

struct ShrinkParams {
    const __nv_bfloat16* x;      // [M][K]
    const float* scale;          // [L] or null (1)
    const int* ids;              // [M]
    int M, K, r, L;
    int passes;                  // CTAs that share a tile's distinct adapters
    int chunks;                  // CTAs along the rank: ceil(r / (8 NT))
    int plan_x;                  // grid columns of the plan
    __nv_bfloat16* tw;           // [M][pairs][r / 8][hi 8 | lo 8]: t 2^-e_m in two bf16 parts
    __half* xh;                  // [M][K]: x 2^-e_m in the dequantizer's k order
    float* rowscale;             // [M]: 2^e_m
    int bits, pairs;
    int* row_slot;               // [M] position of the row's adapter in its token tile's list, or -1
    int* tile_count;             // [num_t] distinct adapters of the token tile
    int* tile_list;              // [num_t][BT] those adapters, in order of first use
    int num_t;
};

// Barrier of the first product's warps.
__device__ __forceinline__ void product_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

// One token tile of the fused kernel: its distinct adapters in order of first use, and each row's place among them.
// A thread takes the rows tid and tid + 128; every row is compared with all of the tile's (no early exit: the loads of
// the loop are then independent), and a place is a count of set bits.
__device__ __forceinline__ void plan_tile(const ShrinkParams& p, int t_blk) {
    constexpr int BT = fused::BT;
    static_assert(BT % 32 == 0 && BT > kThreads && BT <= 2 * kThreads, "one or two rows per thread, whole warps");
    __shared__ __align__(16) int id[BT];
    __shared__ uint32_t leads[BT / 32];            // bit i % 32 of word i / 32: row i is its adapter's first
    const int rows = min(BT, p.M - t_blk * BT);
    for (int i = threadIdx.x; i < BT; i += kThreads) id[i] = i < rows ? adapter_of(p.ids, t_blk * BT + i, p.L) : -1;
    product_sync();
    int first[2];
    const int4* quads = reinterpret_cast<const int4*>(id);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = static_cast<int>(threadIdx.x) + h * kThreads;
        first[h] = i;
        if (i >= BT) continue;                     // whole warps
        const int a = id[i];
#pragma unroll 8
        for (int q = BT / 4 - 1; q >= 0; --q) {
            const int4 v = quads[q];
            first[h] = v.w == a ? 4 * q + 3 : first[h];
            first[h] = v.z == a ? 4 * q + 2 : first[h];
            first[h] = v.y == a ? 4 * q + 1 : first[h];
            first[h] = v.x == a ? 4 * q : first[h];
        }
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, a >= 0 && first[h] == i);
        if ((i & 31) == 0) leads[i >> 5] = bits;
    }
    product_sync();
    const auto place = [&](int i) {                // adapters first met before row i
        int n = 0;
        for (int w = 0; w < BT / 32; ++w) {
            const uint32_t below = w < (i >> 5) ? 0xFFFFFFFFu : w == (i >> 5) ? (1u << (i & 31)) - 1u : 0u;
            n += __popc(leads[w] & below);
        }
        return n;
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = static_cast<int>(threadIdx.x) + h * kThreads;
        if (i >= rows) continue;
        const int n = place(first[h]);
        p.row_slot[t_blk * BT + i] = id[i] >= 0 ? n : -1;
        if (id[i] >= 0 && first[h] == i && in_bounds(n, BT)) p.tile_list[t_blk * BT + n] = id[i];
    }
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < BT / 32; ++w) n += __popc(leads[w]);
        p.tile_count[t_blk] = n;
    }
}

// The conversion's row scale (convert_x_kernel): 2^e with the row's largest magnitude in [2^15, 2^16) after division,
// 1 for a zero or non-finite row.  amax: the largest bf16 bit pattern without its sign.
__device__ __forceinline__ float row_scale(uint32_t amax) {
    const uint32_t ex = amax >> 7;                 // biased exponent
    if (amax == 0 || ex == 0xFF) return 1.0f;
    const int e = max(static_cast<int>(ex) - 127, -100) - 15;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The larger of m and |a|, |b|, per bf16 half; a NaN is passed over, as by the conversion's fmaxf.
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t m, uint32_t a, uint32_t b) {
    uint32_t o;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
    asm("max.bf16x2 %0, %0, %1;" : "+r"(o) : "r"(m));
    return o;
}

// One CTA's part of the first product: the K range of cluster rank `rank` of S, for the tile's n-th distinct adapters
// with n % passes == pass, 8 NT ranks from j0 on, of the pair's member.
//
// Each warp runs a pipeline of its own: its lane 0 keeps kSlots boxes of 32 rows x 64 columns of x, and the same columns
// of the adapter, on their way by TMA while the warp multiplies the oldest (mma.sync, fragments by ldmatrix).  No warp
// waits for another until the sums meet in shared memory, and the cluster's CTAs' in distributed shared memory, each
// added in a fixed order.  t must share the row scale of the converted activations: the rows' maxima are taken from the
// fragments.  Rows of the tile with other adapters are multiplied too and not written.  (The cluster's barriers count
// every live thread: they complete once the converting warps have left.)
template <int NT>
__device__ __forceinline__ void shrink_tile(const CUtensorMap& map_x, const CUtensorMap& map_a, const ShrinkParams& p,
                                            uint8_t* smem, int tile, int pass, int pair, int j0, int rank, int S) {
    constexpr int kSums = kRows * NT * 8;
    constexpr uint32_t kSlot = slot_bytes(NT);
    static_assert(kSums * 4 <= kSlots * kSlot && kSlot % 1024 == 0, "a warp's sums reuse its ring; swizzled boxes");
    __shared__ __align__(8) uint64_t full[kWarps][kSlots];
    __shared__ uint32_t amax[kWarps][kRows];
    __shared__ float scale_s[kRows];
    __shared__ int id_s[kRows];
    __shared__ int abort_flag;
    const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
    const int g = lane >> 2, c = lane & 3;
    const int m0 = tile * kRows;
    const int mine = m0 + lane < p.M ? adapter_of(p.ids, m0 + lane, p.L) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, mine);
    uint32_t leaders = __ballot_sync(0xFFFFFFFFu, mine >= 0 && (__ffs(same) - 1) == lane);
    for (int n = 0; n < pass; ++n) leaders &= leaders - 1;     // the first adapter of this CTA's
    if (warp == 0 && pass == 0 && pair == 0 && j0 == 0 && rank == 0) {
        // rows without an adapter: zeros in tw, so that a tile's boxes of it need no mask
        const int pieces = p.pairs * p.r / 4;
        for (int row = 0; row < kRows && m0 + row < p.M; ++row) {
            if (__shfl_sync(0xFFFFFFFFu, mine, row) >= 0) continue;
            uint4* o = reinterpret_cast<uint4*>(p.tw) + static_cast<int64_t>(m0 + row) * pieces;
            for (int i = lane; i < pieces; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (leaders == 0) return;                                  // the same in every CTA of the cluster
    const int kc_all = p.K / kCols;
    const int kc0 = static_cast<int>(static_cast<int64_t>(kc_all) * rank / S) + warp;          // this warp's first chunk
    const int kc1 = static_cast<int>(static_cast<int64_t>(kc_all) * (rank + 1) / S);
    const int nk = kc0 < kc1 ? (kc1 - kc0 + kWarps - 1) / kWarps : 0;                          // and their number
    uint8_t* ring = smem + warp * kSlots * kSlot;
    const uint32_t ring_addr = ptx::smem_addr(ring);
    float* part = reinterpret_cast<float*>(smem);              // warp w's sums at w * kPartStride
    constexpr int kPartStride = kSlots * kSlot / 4;
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int i = 0; i < kSlots; ++i) ptx::mbar_init(&full[w][i], 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0) id_s[lane] = mine;
    product_sync();
    bool ok = true, first = true;
    uint32_t used = 0, issued = 0;                             // chunks multiplied, copies started (lane 0)
    while (leaders != 0) {
        const int adapter = __shfl_sync(0xFFFFFFFFu, mine, __ffs(leaders) - 1);
        const float factor = p.scale != nullptr ? __ldg(p.scale + adapter) : 1.0f;
        const auto issue = [&](int i) {
            const uint32_t s = issued % kSlots;
            ++issued;
            ptx::mbar_arrive_expect_tx(&full[warp][s], kSlot);
            ptx::tma_load_2d(ring + s * kSlot, &map_x, &full[warp][s], (kc0 + i * kWarps) * kCols, m0);
            ptx::tma_load_3d(ring + s * kSlot + kXSlot, &map_a, &full[warp][s], (kc0 + i * kWarps) * kCols, j0, adapter);
        };
        float acc[2][NT][4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[q][i][e] = 0.0f;
        uint32_t mx[4] = {0u, 0u, 0u, 0u};                     // rows g, g + 8, g + 16, g + 24
        if (lane == 0 && ok && !stalled(kStallPrepare))        // (the checked build can hold every copy back)
            for (int i = 0; i < min(kSlots, nk); ++i) issue(i);
        for (int i = 0; i < nk; ++i, ++used) {
            const uint32_t s = used % kSlots;
            ok = __all_sync(0xFFFFFFFFu, ptx::mbar_wait(&full[warp][s], (used / kSlots) & 1u, &abort_flag)) && ok;
            const uint32_t x_slot = ring_addr + s * kSlot, a_slot = x_slot + kXSlot;
#pragma unroll
            for (int ks = 0; ks < kCols / 16; ++ks) {
                uint32_t xa[2][4], b[(NT + 1) / 2][4];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t row = static_cast<uint32_t>(16 * q + (lane & 15));
                    const uint32_t piece = static_cast<uint32_t>(2 * ks + (lane >> 4));
                    ptx::ldmatrix_x4(x_slot + row * 128 + ((piece ^ (row & 7)) << 4), xa[q]);
                }
#pragma unroll
                for (int j = 0; j < (NT + 1) / 2; ++j) {
                    // two rank blocks: lanes 0-7 and 8-15 address the first one's halves of k, 16-31 the second's
                    const uint32_t row = static_cast<uint32_t>(16 * j + (NT > 1 ? (lane >> 4) * 8 : 0) + (lane & 7));
                    const uint32_t piece = static_cast<uint32_t>(2 * ks + ((lane >> 3) & 1));
                    ptx::ldmatrix_x4(a_slot + row * 128 + ((piece ^ (row & 7)) << 4), b[j]);
                }
                if (first) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        mx[2 * q] = absmax_bf16x2(mx[2 * q], xa[q][0], xa[q][2]);
                        mx[2 * q + 1] = absmax_bf16x2(mx[2 * q + 1], xa[q][1], xa[q][3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        mma_bf16_16816(acc[q][j], xa[q][0], xa[q][1], xa[q][2], xa[q][3], b[j / 2][2 * (j & 1)],
                                       b[j / 2][2 * (j & 1) + 1]);
            }
            __syncwarp();
            if (lane == 0 && ok && i + kSlots < nk) issue(i + kSlots);
        }
        // the warp's ring is empty: its sums go there (after an expired wait: once the copies under way have landed; none
        // is started any more)
        if (!ok && lane == 0) {
            for (uint32_t at = issued > kSlots ? issued - kSlots : 0; at < issued; ++at)
                ptx::mbar_wait(&full[warp][at % kSlots], (at / kSlots) & 1u, nullptr);
            issued = 0;
        }
        __syncwarp();
        float* sums = part + warp * kPartStride;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int at = (16 * q + g) * NT * 8 + 8 * i + 2 * c;
                *reinterpret_cast<float2*>(&sums[at]) = make_float2(acc[q][i][0], acc[q][i][1]);
                *reinterpret_cast<float2*>(&sums[at + 8 * NT * 8]) = make_float2(acc[q][i][2], acc[q][i][3]);
            }
        if (first) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t v = max(mx[q] & 0xFFFFu, mx[q] >> 16);
                v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
                if (c == 0) amax[warp][g + 8 * q] = v;
            }
        }
        product_sync();
        for (int e = threadIdx.x; e < kSums; e += kThreads) {
            float s = part[e];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) s += part[w * kPartStride + e];
            part[e] = s;                                       // this CTA's slice of the sum
        }
        if (first && threadIdx.x < kRows) {
            uint32_t v = amax[0][threadIdx.x];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v = max(v, amax[w][threadIdx.x]);
            amax[0][threadIdx.x] = v;
        }
        if (S > 1) ptx::cluster_sync(); else product_sync();
        if (first) {
            if (threadIdx.x < kRows) {
                uint32_t v = amax[0][threadIdx.x];
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q)
                    if (S > 1 && q < S)
                        v = max(v, __float_as_uint(ptx::ld_shared_cluster_f32(&amax[0][threadIdx.x], static_cast<uint32_t>(q))));
                scale_s[threadIdx.x] = row_scale(v);
            }
            product_sync();
        }
        // every CTA of the cluster finishes its share of the tile's sums, two ranks at a time
        for (int e = 2 * (static_cast<int>(threadIdx.x) + rank * kThreads); e < kSums; e += 2 * S * kThreads) {
            const int row = e / (NT * 8), j = j0 + e % (NT * 8);
            if (j >= p.r || id_s[row] != adapter) continue;
            float s0 = part[e], s1 = part[e + 1];
            if (S > 1) {
                float v0[kMaxSplit], v1[kMaxSplit];            // every CTA's loads before the first sum
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q) {
                    v0[q] = q < S ? ptx::ld_shared_cluster_f32(&part[e], static_cast<uint32_t>(q)) : 0.0f;
                    v1[q] = q < S ? ptx::ld_shared_cluster_f32(&part[e + 1], static_cast<uint32_t>(q)) : 0.0f;
                }
                s0 = v0[0];
                s1 = v1[0];
#pragma unroll
                for (int q = 1; q < kMaxSplit; ++q) {
                    s0 += v0[q];
                    s1 += v1[q];
                }
            }
            // the factor first: s 2^-e_m alone can leave fp32's range where t and t 2^-e_m do not
            const float inv = __uint_as_float(0x7F000000u - __float_as_uint(scale_s[row]));
            const float t0 = s0 * factor * inv, t1 = s1 * factor * inv;
            const int64_t at = (static_cast<int64_t>(m0 + row) * p.pairs + pair) * 2 * p.r + 16 * (j / 8) + j % 8;
            if (!in_bounds(at, static_cast<int64_t>(p.M) * p.pairs * 2 * p.r - 9)) continue;
            *reinterpret_cast<uint32_t*>(p.tw + at) = fused::bf16_part(t0, t1, false);
            *reinterpret_cast<uint32_t*>(p.tw + at + 8) = fused::bf16_part(t0, t1, true);
        }
        first = false;
        for (int n = 0; n < p.passes; ++n) leaders &= leaders - 1;
        // the sums are read, by this CTA and its peers, before the rings are filled again or the CTA ends
        ptx::fence_proxy_async_smem();
        if (S > 1) ptx::cluster_sync(); else product_sync();
    }
}

// The activations' conversion (as convert_x_kernel) of rows first, first + step, ... of the tile, a row by a pair of
// warps: its loads go out together and stay in registers, nine pieces of 8 a thread (4608 columns of a row; the product's
// registers leave no more), and what is beyond is read again from L2.
template <int kBits>
__device__ __forceinline__ void convert_rows(const ShrinkParams& p, int m0, int first, int step, int group) {
    __shared__ float red[2][kConvGroups][2];
    constexpr int kCache = 9;
    const int tid = static_cast<int>(threadIdx.x - kThreads) & (kConvThreads - 1);
    const int n8 = p.K / 8;
    int parity = 0;
    for (int row = first; row < kRows && m0 + row < p.M; row += step, parity ^= 1) {
        const uint4* src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(m0 + row) * p.K);
        uint4* dst = reinterpret_cast<uint4*>(p.xh + static_cast<int64_t>(m0 + row) * p.K);
        uint4 v[kCache];
#pragma unroll
        for (int j = 0; j < kCache; ++j) {
            const int i = tid + j * kConvThreads;
            v[j] = i < n8 ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        }
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < kCache; ++j) top = absmax_bf16x8(v[j], top);
#pragma unroll 2
        for (int i = tid + kCache * kConvThreads; i < n8; i += kConvThreads) top = absmax_bf16x8(__ldg(src + i), top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        if ((tid & 31) == 0) red[parity][group][tid >> 5] = top;
        asm volatile("bar.sync %0, %1;" ::"r"(2 + group), "n"(kConvThreads) : "memory");
        top = fmaxf(red[parity][group][0], red[parity][group][1]);
        const float sc = row_scale(__float_as_uint(top) >> 16);
        if (tid == 0) p.rowscale[m0 + row] = sc;
        const float inv = __uint_as_float(0x7F000000u - __float_as_uint(sc));
#pragma unroll
        for (int j = 0; j < kCache; ++j) {
            const int i = tid + j * kConvThreads;
            if (i < n8) dst[i] = convert8<kBits>(v[j], inv);
        }
#pragma unroll 2
        for (int i = tid + kCache * kConvThreads; i < n8; i += kConvThreads) dst[i] = convert8<kBits>(__ldg(src + i), inv);
    }
}

// Everything the adapters of a fused call need before the GEMM, in one launch: the token tiles' adapter lists, the
// activations' conversion and the adapters' first product.  grid (plan_x + tiles * passes * chunks * pairs, S), cluster
// (1, S, 1): first the lists, then the CTAs of every tile of 32 rows.  A tile's first column of CTAs also converts its
// rows, in warps of their own beside the product's, so that the two readers of a row meet in L2 (33792 x 4608, rank 32:
// 408 MB read from DRAM for 311 MB of x).  What passes between L2 and the SMs there is x twice, its converted copy and A
// once per tile, 1.24 GB in 162 us; neither DRAM nor L2 is near its rate (a fifth and a third of it), each warp waits for
// its own three boxes.  With few tiles it is latency: 18 us for 333 rows.  (One kernel after the other read x from DRAM
// twice, 182 us; both by the same warps, the tile held in shared memory between product and conversion, spent its time in
// one tile's barriers, 265 us.)  Two CTAs per SM leave 80 registers a thread; 31 to 35 are spilled.
template <int NT>
__global__ void __launch_bounds__(kBlock, 2) lora_prepare_kernel(const __grid_constant__ CUtensorMap map_x,
                                                                 const __grid_constant__ CUtensorMap map_a0,
                                                                 const __grid_constant__ CUtensorMap map_a1,
                                                                 const ShrinkParams p) {
    ptx::launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    const int S = static_cast<int>(gridDim.y), rank = static_cast<int>(blockIdx.y);            // rank in the cluster
    const int bx = static_cast<int>(blockIdx.x) - p.plan_x;
    const int products = p.passes * p.chunks * p.pairs;
    const int tile = bx / products, i = bx - tile * products;
    if (threadIdx.x >= kThreads) {
        if (bx < 0 || i != 0) return;
        test_delay(kDelayActivations);   // the checked build can hold these warps back (qlinear_test_delay)
        const int group = static_cast<int>(threadIdx.x - kThreads) / kConvThreads;
        if (p.bits == 4) convert_rows<4>(p, tile * kRows, rank + S * group, S * kConvGroups, group);
        else convert_rows<8>(p, tile * kRows, rank + S * group, S * kConvGroups, group);
        return;
    }
    test_delay(bx < 0 ? kDelayCodes : kDelayMma);   // (and the lists', the product's)
    if (bx < 0) {
        const int t_blk = static_cast<int>(blockIdx.x) * S + rank;
        if (t_blk < p.num_t) plan_tile(p, t_blk);
    } else {
        const int pass = i % p.passes, chunk = i / p.passes % p.chunks, pair = i / p.passes / p.chunks;
        uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
        shrink_tile<NT>(map_x, pair == 0 ? map_a0 : map_a1, p, smem, tile, pass, pair, chunk * NT * 8, rank, S);
    }
    // Launched behind the parameter transpose under programmatic dependent launch; as with the conversion of the
    // plain layer, the last CTA waits for it, so that this kernel's completion implies both.
    if (blockIdx.x == gridDim.x - 1) ptx::grid_dependency_wait();
}

// The weight-streaming path's last kernel: y[t][n] = 2^rowexp[t] * (sum of the stream-K partials, as
// skinny_reduce_kernel) + sum_j t[t][j] B[a][n][j] with t = s sum_z tp[z], all in fp32 from the bf16 adapter, rounded
// once.  kPair: g and u of a gate/up pair that way, from the two tiles of the column, and h = silu(g) u.  A CTA takes a
// 128-column tile and two tokens at a time, the tokens y, y + gridDim.y, ... of the pairs of tokens: listing the tile's
// partials once for many tokens, in one wave of CTAs (24 tokens x 12288 pairs: 10 us behind the stream, of which the CTAs'
// start takes 4; one token's 13824 columns 2.7 us).  The first tokens' B is loaded before the wait for the partials.
struct ExpandParams {
    const __nv_bfloat16* b[2];   // [L][N][r] of each member
    const float* scale;          // [L] or null (1)
    const float* tp;             // [slices][pairs][M][r]
    const int* ids;              // [M]
    int r, L, slices;
};

template <bool kBf16Out, bool kPair>
__global__ void __launch_bounds__(256) lora_reduce_kernel(const float* __restrict__ partial,
                                                          const int* __restrict__ rowexp, void* __restrict__ y, int M,
                                                          int N, int cpt, int64_t units, int P, int segmax,
                                                          int64_t partial_elems, const ExpandParams ep) {
    constexpr int kPairs = kPair ? 2 : 1;
    constexpr int kEager = kPair ? 2 : 4;
    __shared__ int64_t seg_base[kPairs][skinny::kMaxCtas];
    __shared__ int count[kPairs];
    __shared__ float ps[2][kPairs][128];
    __shared__ __align__(16) float tl[2][kPairs][kMaxRank];
    const int w = blockIdx.x;                                     // tile of the gate weight; the up's is w + gridDim.x
    const int half = threadIdx.x >> 7, i128 = threadIdx.x & 127;
    const int n = w * skinny::BW + i128;
    const int step = 2 * static_cast<int>(gridDim.y);
    const int groups = 128 / ep.r, j = i128 % ep.r, group = i128 / ep.r;
    const auto adapter = [&](int t) {                             // the first product records an id out of range
        const int a = t < M ? ep.ids[t] : -1;
        return a < ep.L ? a : -1;
    };
    int t = blockIdx.y * 2 + half;
    int a = adapter(t);
    if (i128 == 0 && half < kPairs)
        count[half] = skinny::list_segments(w + half * static_cast<int>(gridDim.x), cpt, units, P, segmax, seg_base[half]);
    bool first = true;
    for (int t0 = blockIdx.y * 2; t0 < M; t0 += step, t += step) {
        const bool live = t < M && n < N, with = a >= 0;
        const int chunks = with && live ? ep.r / 8 : 0;
        const int64_t row = (static_cast<int64_t>(with ? a : 0) * N + (live ? n : 0)) * ep.r;
        uint4 eager[kPairs][kEager];
#pragma unroll
        for (int q = 0; q < kPairs; ++q)
#pragma unroll
            for (int i = 0; i < kEager; ++i)
                eager[q][i] = i < chunks ? __ldg(reinterpret_cast<const uint4*>(ep.b[q] + row) + i) : make_uint4(0u, 0u, 0u, 0u);
        const float sc = with && ep.scale != nullptr ? __ldg(ep.scale + a) : 1.0f;
        __syncthreads();                                          // the lists are complete; ps and tl are free
        if (first) ptx::grid_dependency_wait();                   // partials and tp come from the kernel before
        first = false;
        // t of the two tokens: a token's 128 threads share out the slices, then add their sums in order
        if (with && group < groups) {
            const int64_t stride = static_cast<int64_t>(kPairs) * M * ep.r;
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                const float* tp = ep.tp + (static_cast<int64_t>(q) * M + t) * ep.r + j;
                float sum = 0.0f;
#pragma unroll 8
                for (int z = group; z < ep.slices; z += groups) sum += tp[z * stride];
                ps[half][q][i128] = sum;
            }
        }
        float acc[kPairs];
#pragma unroll
        for (int q = 0; q < kPairs; ++q)
            acc[q] = live ? skinny::sum_segments(partial, partial_elems, seg_base[q], count[q], M, t, i128) : 0.0f;
        const int ex = live ? rowexp[t] : 0;
        __syncthreads();
        if (with && i128 < ep.r) {
#pragma unroll
            for (int q = 0; q < kPairs; ++q) {
                float sum = ps[half][q][i128];
                for (int z = 1; z < groups; ++z) sum += ps[half][q][i128 + z * ep.r];
                tl[half][q][i128] = sc * sum;
            }
        }
        a = adapter(t + step);
        __syncthreads();
        if (!live) continue;                                      // back to the first barrier, like every thread
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
            const float4* tt = reinterpret_cast<const float4*>(tl[half][q]);
            const uint4* b = reinterpret_cast<const uint4*>(ep.b[q] + row);
            float delta = 0.0f;
            const auto add = [&](const uint4 v, int i) {
                const float4 t0 = tt[2 * i], t1 = tt[2 * i + 1];
                delta = fmaf(t0.x, bf16_lo(v.x), delta);
                delta = fmaf(t0.y, bf16_hi(v.x), delta);
                delta = fmaf(t0.z, bf16_lo(v.y), delta);
                delta = fmaf(t0.w, bf16_hi(v.y), delta);
                delta = fmaf(t1.x, bf16_lo(v.z), delta);
                delta = fmaf(t1.y, bf16_hi(v.z), delta);
                delta = fmaf(t1.z, bf16_lo(v.w), delta);
                delta = fmaf(t1.w, bf16_hi(v.w), delta);
            };
#pragma unroll
            for (int i = 0; i < kEager; ++i)
                if (i < chunks) add(eager[q][i], i);
#pragma unroll 1
            for (int i = kEager; i < chunks; ++i) add(__ldg(b + i), i);
            if (!(fabsf(delta) <= 3.4028235e38f)) {
                // rare: a non-finite entry of B (then it counts as zero and is recorded, as on the fused path), or t
                delta = 0.0f;
#pragma unroll 1
                for (int i = 0; i < chunks; ++i) {
                    const uint4 v = __ldg(b + i);
                    add(make_uint4(finite_bf16x2(v.x), finite_bf16x2(v.y), finite_bf16x2(v.z), finite_bf16x2(v.w)), i);
                }
            }
            acc[q] = ldexpf(acc[q], ex) + delta;
        }
        float out = acc[0];
        // as the fused kernel's SwiGLU epilogue
        if constexpr (kPair) out = __fdividef(acc[0], 1.0f + __expf(-acc[0])) * acc[1];
        const int64_t e = static_cast<int64_t>(t) * N + n;
        if constexpr (kBf16Out) {
            reinterpret_cast<__nv_bfloat16*>(y)[e] = __float2bfloat16_rn(out);
        } else {
            reinterpret_cast<float*>(y)[e] = out;
        }
    }
}

}  // namespace lora
}  // namespace ql
