// The norms after and before a block, fused with its gate and the residual update between them.
//
//   v = sum_z y[z]                                    the block's output: bf16, or fp32 partials [S] in order
//   v = v / sqrt(mean_d v^2 + eps) * post_weight      (post norm, optional)
//   r = residual_scale * x + branch_scale * gate[seg] * v
//   h = r / sqrt(mean_d r^2 + eps) * pre_weight * (1 + scale[seg]) + shift[seg]      (pre norm, optional)
//
// Without y, r is x itself and only h is written.  Everything between the loads and the two stores is fp32;
// r and h are rounded once each, and h is formed from the unrounded r.  A row whose segment is negative is
// padding: nothing of it is read or written.
//
// The operation moves each row once and does a dozen flops per element, so DRAM bounds it; a row therefore
// stays in registers from its load to its stores.  The vectors (weights, gate, scale, shift) are read
// through L1, where the rows of one SM share them.  Rows of up to kWarpRowMax elements take one warp each
// (no block barrier); longer rows take a CTA with up to kMaxVec 8-element vectors per thread.
#pragma once

#include "ql_ptx.cuh"

namespace ql {
namespace norm {

constexpr int kMaxD = 32768;          // 1024 threads x 4 vectors of 8
constexpr int kWarpRowMax = 1024;     // 32 lanes x 4 vectors of 8
constexpr int kWarpRows = 4;          // rows (warps) per CTA of the warp-per-row form

enum { kYNone = 0, kYBf16 = 1, kYF32 = 2 };

struct Params {
    const void* x;             // [M][D] TX
    const void* y;             // [M][D] bf16, or fp32 [S][M][D]
    void* r;                   // [M][D] TX, may be x
    __nv_bfloat16* h;          // [M][D], or null
    const void* post_weight;   // [D] or null (1)
    const void* gate;          // [T][D] or null (1)
    const void* pre_weight;    // [D] or null (1)
    const void* scale;         // [T][D] or null (0)
    const void* shift;         // [T][D] or null (0)
    const int* seg;            // [M] or null (segment 0)
    int64_t M;
    int D, S, T;
    int params_f32;            // the vectors' type: 0 bf16, 1 fp32
    int post_norm;
    float residual_scale, branch_scale, eps;
};

// Rows are read once: keep them out of L1, which holds the vectors.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void unpack_f32x8(const uint4 a, const uint4 b, float (&f)[8]) {
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
}

// 8 elements of a parameter vector from element i on.
__device__ __forceinline__ void load_params(const void* p, int f32, int64_t i, float (&f)[8]) {
    if (f32) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        unpack_f32x8(__ldg(q), __ldg(q + 1), f);
    } else {
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)), f);
    }
}

template <bool kF32>
__device__ __forceinline__ void load_row(const void* p, int64_t i, float (&f)[8]) {
    if constexpr (kF32) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        const uint4 a = ld_stream(q), b = ld_stream(q + 1);
        unpack_f32x8(a, b, f);
    } else {
        unpack_bf16x8(ld_stream(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)), f);
    }
}

// Sum of v over the row's threads (a warp, or the CTA through one shared float per warp), in a fixed order.
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (kWarpRow) return v;
    const int nwarps = static_cast<int>(blockDim.x >> 5);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = static_cast<int>(threadIdx.x & 31) < nwarps ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}

template <bool kXF32, int kY, int VPT, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 32 * kWarpRows : 1024) norm_residual_kernel(const Params p) {
    __shared__ float red[2][32];
    const int tid = kWarpRow ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
    const int nthreads = kWarpRow ? 32 : static_cast<int>(blockDim.x);
    const int64_t m = kWarpRow ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (m >= p.M) return;
    int seg = 0;
    if (p.seg != nullptr) {
        seg = p.seg[m];
        if (seg >= p.T) {
            if (tid == 0) record_status(QL_ERR_INVALID_ARG);
            return;
        }
        if (seg < 0) return;                           // padding
    }
    const int D = p.D, nv = D / 8;
    const int64_t row = m * D;
    const int64_t vec = static_cast<int64_t>(seg) * D;
    const float inv_d = 1.0f / static_cast<float>(D);

    float r[VPT][8];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = tid + j * nthreads;
#pragma unroll
        for (int k = 0; k < 8; ++k) r[j][k] = 0.0f;
        if (c < nv) load_row<kXF32>(p.x, row + 8 * c, r[j]);
    }
    if constexpr (kY != kYNone) {
        float v[VPT][8];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid + j * nthreads;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[j][k] = 0.0f;
            if (c < nv) load_row<kY == kYF32>(p.y, row + 8 * c, v[j]);
        }
        if constexpr (kY == kYF32) {
            for (int z = 1; z < p.S; ++z) {
                const int64_t at = (static_cast<int64_t>(z) * p.M) * D + row;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int c = tid + j * nthreads;
                    float w[8];
                    if (c < nv) {
                        load_row<true>(p.y, at + 8 * c, w);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[j][k] += w[k];
                    }
                }
            }
        }
        float inv = 1.0f;
        if (p.post_norm) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < VPT; ++j)
#pragma unroll
                for (int k = 0; k < 8; ++k) ss = fmaf(v[j][k], v[j][k], ss);
            inv = 1.0f / sqrtf(row_sum<kWarpRow>(ss, red[0]) * inv_d + p.eps);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid + j * nthreads;
            if (c >= nv) continue;
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[j][k] *= inv;
            if (p.post_weight != nullptr) {
                load_params(p.post_weight, p.params_f32, 8 * c, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[j][k] *= f[k];
            }
            if (p.gate != nullptr) {
                load_params(p.gate, p.params_f32, vec + 8 * c, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[j][k] *= f[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) r[j][k] = fmaf(p.branch_scale, v[j][k], p.residual_scale * r[j][k]);
            if constexpr (kXF32) {
                float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.r) + row + 8 * c);
                o[0] = make_float4(r[j][0], r[j][1], r[j][2], r[j][3]);
                o[1] = make_float4(r[j][4], r[j][5], r[j][6], r[j][7]);
            } else {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.r) + row + 8 * c) = pack_bf16x8(r[j]);
            }
        }
    }
    if (p.h == nullptr) return;
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(r[j][k], r[j][k], ss);     // threads past the row's end hold zeros
    const float inv = 1.0f / sqrtf(row_sum<kWarpRow>(ss, red[1]) * inv_d + p.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = tid + j * nthreads;
        if (c >= nv) continue;
        float f[8], o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = r[j][k] * inv;
        if (p.pre_weight != nullptr) {
            load_params(p.pre_weight, p.params_f32, 8 * c, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] *= f[k];
        }
        if (p.scale != nullptr) {
            load_params(p.scale, p.params_f32, vec + 8 * c, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = fmaf(o[k], f[k], o[k]);
        }
        if (p.shift != nullptr) {
            load_params(p.shift, p.params_f32, vec + 8 * c, f);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] += f[k];
        }
        *reinterpret_cast<uint4*>(p.h + row + 8 * c) = pack_bf16x8(o);
    }
}

}  // namespace norm
}  // namespace ql
