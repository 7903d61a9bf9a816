// A packed projection of a few tokens (up to 32) with its epilogue, in one launch.
//
//   y[m][n] = epilogue( sum_g s(n,g) D(n,m,g) + (b(n,g) - 128 s(n,g)) X(m,g) )
//   D = sum_{k in g} (128 + q(n,k)) x[m][k],   X = sum_{k in g} x[m][k]
//
// which is sum_k (s q + b) x, rearranged by group: 128 + q, for a code of 4 bits, is the bf16 whose mantissa holds q, so a
// pair of weights takes a shift and one logical operation, and the activations are used as they are.  The tensor core
// (mma m16n8k16, 16 weight rows x 8 tokens, fp32) sums a group's products exactly up to its own fp32 additions; X comes
// from the same operands times ones.  8-bit codes are two nibbles, q = 16 h + l, of a product each.
//
// What bounds such a call is not the 0.56 bytes a weight that it reads but the launches: the streaming path's conversion,
// stream and reduction, three kernels, take 11.7 us for 1 token of 4608 x 4608 whose 12 MB come from memory (1.8 us at its
// rate), this one 8.0 (from L2 11.1 and 7.1).  Its weights are exact, not rounded to f16 as the other paths' are.  A warp
// takes 16 rows and a slice of their groups; the warps of a CTA that share rows add up in shared memory, in order.  (With
// the groups dealt out in turn, a request for each scale, it took 8.1 from L2: every request touches eight rows' lines.)
#pragma once

#include "ql_epilogue.cuh"

namespace ql {
namespace few {

constexpr int kMaxM = 32;              // four blocks of 8 tokens
constexpr int kWarps = 8;
constexpr int kRows = 16;              // of a warp
constexpr int kAhead = 4;              // groups whose loads are on their way together

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 128 + q for the two codes of 4 bits at bits 0 and 16.
__device__ __forceinline__ uint32_t weights_of(uint32_t v) { return (v & 0x000F000Fu) | 0x43004300u; }

// Lane l = 4 r + t of a warp holds, of weight rows r and r + 8 and of tokens r, r + 8, .., the 16 columns 16 t .. of a
// group: which of a product's 16 columns an operand's register stands for is free as long as both operands agree.
template <int B>
struct Codes {
    uint32_t w[2][B == 4 ? 2 : 4];     // of rows r, r + 8
};
template <int NT>
struct Tokens {
    uint4 x[NT][2];
};

// NT: blocks of 8 tokens.
template <int B, int NT, bool kBf16Out>
__global__ void __launch_bounds__(32 * kWarps) few_kernel(const __nv_bfloat16* __restrict__ x, const uint32_t* __restrict__ codes,
                                                          const unsigned short* __restrict__ scales,
                                                          const unsigned short* __restrict__ biases, void* y, int M, int K, int N,
                                                          int slices, const epi::Epilogue e) {
    __shared__ float red[kWarps][8 * NT][kRows];
    const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
    const int r = lane >> 2, t = lane & 3;
    const int G = K / kGroup, slice = warp % slices, block = warp / slices;
    const int blocks = kWarps / slices;                // of 16 rows per CTA
    const int n0 = (static_cast<int>(blockIdx.x) * blocks + block) * kRows;
    constexpr int kWords = B == 4 ? 2 : 4;             // a lane's, of a row's group

    const auto load = [&](int g, Codes<B>& o) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t n = min(n0 + r + 8 * h, N - 1);              // (rows past N are not stored)
            const int64_t at = n * (K * B / 32) + g * (2 * B) + kWords * t;
            const uint32_t* c = codes + at;
            if (!in_bounds(at + kWords - 1, static_cast<int64_t>(N) * (K * B / 32))) {
                o = {};
                continue;
            }
            if constexpr (B == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(c));
                o.w[h][0] = v.x;
                o.w[h][1] = v.y;
            } else {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(c));
                o.w[h][0] = v.x;
                o.w[h][1] = v.y;
                o.w[h][2] = v.z;
                o.w[h][3] = v.w;
            }
        }
    };
    const auto load_x = [&](int g, Tokens<NT>& o) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            o.x[i][0] = o.x[i][1] = make_uint4(0u, 0u, 0u, 0u);
            const int64_t at = static_cast<int64_t>(r + 8 * i) * K + g * kGroup + 16 * t;
            if (r + 8 * i < M && in_bounds(at + 15, static_cast<int64_t>(M) * K)) {
                const uint4* v = reinterpret_cast<const uint4*>(x + at);
                o.x[i][0] = __ldg(v);
                o.x[i][1] = __ldg(v + 1);
            }
        }
    };
    float acc[NT][4] = {};                             // rows r, r, r + 8, r + 8 of tokens 2 t, 2 t + 1, ... of a block
    const auto work = [&](const Codes<B>& o, const Tokens<NT>& xs, const uint32_t (&sb)[2], int i4) {
        float s[2], b[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2 p = half2_of(__shfl_sync(0xFFFFFFFFu, sb[h], 4 * r + i4));
            s[h] = __low2float(p);
            b[h] = fmaf(s[h], B == 4 ? -128.0f : -17.0f * 128.0f, __high2float(p));
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (NT > 1 && 8 * j >= M) break;
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, hi[4] = {0.0f, 0.0f, 0.0f, 0.0f}, one[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            constexpr uint32_t kOnes = 0x3F803F80u;
            const uint4 x0 = xs.x[j][0], x1 = xs.x[j][1];
            const uint32_t xw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t b0, b1;
                if constexpr (B == 4) {
                    // word u / 2 of each row, its code pairs (k, k + 4) for k = 2 (u % 2) and + 1
                    const uint32_t lo = xw[4 * (u >> 1) + (u & 1)], up = xw[4 * (u >> 1) + 2 + (u & 1)];
                    b0 = __byte_perm(lo, up, 0x5410);
                    b1 = __byte_perm(lo, up, 0x7632);
                    const uint32_t p = o.w[0][u >> 1] >> (8 * (u & 1)), q = o.w[1][u >> 1] >> (8 * (u & 1));
                    mma_bf16(d, weights_of(p), weights_of(q), weights_of(p >> 4), weights_of(q >> 4), b0, b1);
                } else {
                    // word u of each row, its code pairs (0, 2) and (1, 3), by nibbles
                    b0 = __byte_perm(xw[2 * u], xw[2 * u + 1], 0x5410);
                    b1 = __byte_perm(xw[2 * u], xw[2 * u + 1], 0x7632);
                    const uint32_t p = o.w[0][u], q = o.w[1][u];
                    mma_bf16(d, weights_of(p), weights_of(q), weights_of(p >> 8), weights_of(q >> 8), b0, b1);
                    mma_bf16(hi, weights_of(p >> 4), weights_of(q >> 4), weights_of(p >> 12), weights_of(q >> 12), b0, b1);
                }
                mma_bf16(one, kOnes, kOnes, kOnes, kOnes, b0, b1);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = B == 4 ? d[i] : fmaf(16.0f, hi[i], d[i]);
                acc[j][i] = fmaf(s[i >> 1], v, fmaf(b[i >> 1], one[i], acc[j][i]));
            }
        }
    };
    // The slice's groups four at a time, the codes of the four on their way before the first is used; the activations too
    // where they are one block's, else a group ahead.  Lane t of a row's four takes the (scale, bias) of the t-th group:
    // one request instead of four, each of which touches eight rows' lines.
    static_assert(kAhead == 4, "a group for each lane of a row's four");
    const int g_end = static_cast<int>(static_cast<int64_t>(slice + 1) * G / slices);
    constexpr int kAheadX = NT == 1 ? kAhead : 2;
    for (int g = static_cast<int>(static_cast<int64_t>(slice) * G / slices); g < g_end; g += kAhead) {
        Codes<B> o[kAhead];
        Tokens<NT> xs[kAheadX];
        uint32_t sb[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = static_cast<int64_t>(min(n0 + r + 8 * h, N - 1)) * G + min(g + t, g_end - 1);
            sb[h] = 0u;
            if (in_bounds(at, static_cast<int64_t>(N) * G))
                sb[h] = __ldg(scales + at) | static_cast<uint32_t>(__ldg(biases + at)) << 16;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (g + i < g_end) load(g + i, o[i]);
            if (i < kAheadX && g + i < g_end) load_x(g + i, xs[i]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (g + i < g_end) work(o[i], xs[i % kAheadX], sb, i);
            if (NT > 1 && i + kAheadX < kAhead && g + i + kAheadX < g_end) load_x(g + i + kAheadX, xs[i % kAheadX]);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[warp][8 * j + 2 * t + (i & 1)][r + 8 * (i >> 1)] = acc[j][i];
    __syncthreads();
    // the outputs of a row block: kRows rows of every token, summed over the slices in order
    for (int i = static_cast<int>(threadIdx.x); i < blocks * M * kRows; i += 32 * kWarps) {
        const int row = i % kRows, m = i / kRows % M, bl = i / (kRows * M);
        const int n = (static_cast<int>(blockIdx.x) * blocks + bl) * kRows + row;
        if (n >= N) continue;
        const int seg = epi::segment_of(e, m, M);
        if (seg < 0) continue;
        float z = epi::bias_of(e, N, n), sum = 0.0f;
        for (int s = 0; s < slices; ++s) sum += red[bl * slices + s][m][row];
        z += sum;
        const int64_t at = static_cast<int64_t>(m) * N + n;
        if (!in_bounds(at, static_cast<int64_t>(M) * N)) continue;
        const float gate = epi::gate_of(e, seg, N, n);
        float res = 0.0f;
        if (e.residual != nullptr)
            res = kBf16Out ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[at])
                           : static_cast<const float*>(e.residual)[at];
        const float o = fmaf(gate, epi::activate(e.act, z), res);
        if constexpr (kBf16Out)
            static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(o);
        else
            static_cast<float*>(y)[at] = o;
    }
}

}  // namespace few
}  // namespace ql
