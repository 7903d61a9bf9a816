// What follows a packed projection, in its epilogue:
//
//   z = x . W^T + bias[n]
//   a = act(z)                            none, silu, gelu or its tanh form
//   y = residual + gate[seg[m]][n] * a    fp32 from the accumulator on, rounded once
//
// A row whose segment is negative is padding: its row of y is left as it was.
#pragma once

#include "ql_norm.cuh"
#include "ql_ptx.cuh"
#include "ql_tc_skinny.cuh"

namespace ql {
namespace epi {

struct Epilogue {
    const void* bias;        // [N] or null (0)
    const void* gate;        // [T][N] or null (1)
    const void* residual;    // [M][N] of y's type, may be y, or null (0)
    const int* seg;          // [M] or null (segment 0)
    int T;
    int act;                 // ql_activation
    int params_f32;          // type of bias and gate: 0 bf16, 1 fp32
};

// The hardware's base-2 exponential (relative error 2^-22) and reciprocal (2^-23).  Rounding the exponential's argument adds
// its magnitude times a few 2^-24, so that the activations below keep their relative accuracy in their tails, (20 + 8 E) 2^-24
// of the value where e^-E is the exponential.  Results under 2^-120 may come out as zero.
__device__ __forceinline__ float exp2_fast(float v) {
    float o;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
    return o;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float o;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
    return o;
}
constexpr float kLog2e = 1.44269504f;

// z / (1 + e^-z); where e^-z overflows the reciprocal is 0 and the result -0.
__device__ __forceinline__ float silu(float z) { return z * rcp_fast(1.0f + exp2_fast(-kLog2e * z)); }

// z Phi(z), where 1 - Phi(|z|) = t P(t) e^(-z^2 / 2), t = 1 / (1 + 0.35 |z|): the form of Abramowitz and Stegun, Handbook of
// Mathematical Functions, 7.1.26, with P of degree 6 fitted (minimax over 0 <= |z| <= 13.5, by linear programming) to the
// relative error, which stays under 2^-22 (1 + z^2 / 2).  Their five terms keep 1.5e-7 of 1, but only 0.2 % of the tail itself
// at z = -5 and 1 % at -8.  The library's erff takes some forty instructions and a branch, this takes sixteen.
__device__ __forceinline__ float gelu(float z) {
    const float t = rcp_fast(fmaf(0.35f, fabsf(z), 1.0f));
    const float p = fmaf(t, fmaf(t, fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.045832973f, -0.18913298f), 0.21832183f), 0.0033125462f),
                                          0.14543160f), 0.13642566f), 0.13980844f);
    const float tail = t * p * exp2_fast(-0.5f * kLog2e * z * z);      // 1 - Phi(|z|)
    // z - z tail above zero, z tail below (an infinite z times a zero tail would be NaN)
    return fmaf(-fminf(fabsf(z), 1e4f), tail, fmaxf(z, 0.0f));
}
// The same for two values, to the same bits: packed operations where there are some.  The fused kernel's drain is bound by
// its instructions there: 4608 x 128 x 4608 39 us instead of 44 (41 with the five terms of 7.1.26).
__device__ __forceinline__ float2 gelu_pair(float z0, float z1) {
    using norm::fma2, norm::mul2, norm::pair_of, norm::halves;
    const auto both = [](float v) { return pair_of(v, v); };
    const uint64_t t = pair_of(rcp_fast(fmaf(0.35f, fabsf(z0), 1.0f)), rcp_fast(fmaf(0.35f, fabsf(z1), 1.0f)));
    uint64_t p = fma2(t, both(0.045832973f), both(-0.18913298f));
    p = fma2(t, p, both(0.21832183f));
    p = fma2(t, p, both(0.0033125462f));
    p = fma2(t, p, both(0.14543160f));
    p = fma2(t, p, both(0.13642566f));
    p = fma2(t, p, both(0.13980844f));
    const uint64_t z = pair_of(z0, z1);
    const float2 v = halves(mul2(mul2(both(-0.5f * kLog2e), z), z));
    const float2 tail = halves(mul2(mul2(t, p), pair_of(exp2_fast(v.x), exp2_fast(v.y))));
    return make_float2(fmaf(-fminf(fabsf(z0), 1e4f), tail.x, fmaxf(z0, 0.0f)),
                       fmaf(-fminf(fabsf(z1), 1e4f), tail.y, fmaxf(z1, 0.0f)));
}

// 0.5 z (1 + tanh(u)) = z / (1 + e^-2u), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu_tanh(float z) {
    const float u = z * fmaf(0.044715f * 1.59576912f * -kLog2e, z * z, 1.59576912f * -kLog2e);    // -2 u log2(e)
    return z * rcp_fast(1.0f + exp2_fast(u));
}

template <int kAct>
__device__ __forceinline__ float activate_as(float z) {
    return kAct == QL_ACT_SILU ? silu(z) : kAct == QL_ACT_GELU ? gelu(z) : kAct == QL_ACT_GELU_TANH ? gelu_tanh(z) : z;
}
template <int kAct>
__device__ __forceinline__ float2 activate_as(float z0, float z1) {
    if constexpr (kAct == QL_ACT_GELU) return gelu_pair(z0, z1);
    return make_float2(activate_as<kAct>(z0), activate_as<kAct>(z1));
}
__device__ __forceinline__ float activate(int act, float z) {
    switch (act) {
        case QL_ACT_SILU: return silu(z);
        case QL_ACT_GELU: return gelu(z);
        case QL_ACT_GELU_TANH: return gelu_tanh(z);
        default: return z;
    }
}

// Segment of row m of M, -1 for a row to leave alone.
__device__ __forceinline__ int segment_of(const Epilogue& e, int64_t m, int64_t M) {
    if (e.seg == nullptr) return 0;
    if (!in_bounds(m, M)) return -1;
    const int s = __ldg(e.seg + m);
    if (s >= e.T) {
        record_status(QL_ERR_INVALID_ARG);
        return -1;
    }
    return s < 0 ? -1 : s;
}

__device__ __forceinline__ float param(const void* p, int f32, int64_t i) {
    return f32 ? __ldg(static_cast<const float*>(p) + i)
               : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}
// Bias and gate of column n of N; 0 and 1 where there is none.
__device__ __forceinline__ float bias_of(const Epilogue& e, int64_t N, int64_t n) {
    return e.bias != nullptr && in_bounds(n, N) ? param(e.bias, e.params_f32, n) : 0.0f;
}
__device__ __forceinline__ float gate_of(const Epilogue& e, int seg, int64_t N, int64_t n) {
    return e.gate != nullptr && in_bounds(seg * N + n, e.T * N) ? param(e.gate, e.params_f32, seg * N + n) : 1.0f;
}
__device__ __forceinline__ float4 bf16x4(uint2 v) {
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
__device__ __forceinline__ float4 param4(const void* p, int f32, int64_t i) {
    return f32 ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i))
               : bf16x4(__ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i)));
}

// y = epilogue of the fp32 partials [S][M][N], summed in slice order: four columns per thread, whose bias (and gate,
// while the segment stays the same) it holds over its rows.  What the caller gave of a row is fetched a row ahead, of the
// first one before the wait for the partials (its chain begins with a plain launch, see launch_epilogue_sum).
template <bool kBf16Out>
__global__ void __launch_bounds__(256) epilogue_sum_kernel(const float* __restrict__ partial, void* y, int64_t M, int N,
                                                           int S, const Epilogue e) {
    const int n = 4 * static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x);
    if (n >= N) return;
    const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float4 gate = make_float4(1.0f, 1.0f, 1.0f, 1.0f), r_next = none;
    int held = -1, seg_next = -1;
    const auto fetch = [&](int64_t m) {
        if (m >= M) return;
        seg_next = segment_of(e, m, M);
        const int64_t at = m * N + n;
        if (e.residual == nullptr || !in_bounds(at + 3, M * N)) return;
        r_next = kBf16Out ? bf16x4(*reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(e.residual) + at))
                          : *reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + at);
    };
    const float4 bias = e.bias && in_bounds(n + 3, N) ? param4(e.bias, e.params_f32, n) : none;
    fetch(blockIdx.y);
    ptx::grid_dependency_wait();                       // the partials come from the kernel before
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        const int seg = seg_next;
        const float4 r = r_next;
        const int64_t at = m * N + n;
        fetch(m + gridDim.y);
        if (seg < 0) continue;
        if (e.gate != nullptr && seg != held && in_bounds(static_cast<int64_t>(seg) * N + n + 3, static_cast<int64_t>(e.T) * N))
            gate = param4(e.gate, e.params_f32, static_cast<int64_t>(seg) * N + n);
        held = seg;
        float4 z = none;
#pragma unroll 4
        for (int s = 0; s < S; ++s) {
            if (!in_bounds(s * M * N + at + 3, S * M * N)) continue;
            const float4 v = *reinterpret_cast<const float4*>(partial + s * M * N + at);
            z = make_float4(z.x + v.x, z.y + v.y, z.z + v.z, z.w + v.w);
        }
        const float4 o = make_float4(fmaf(gate.x, activate(e.act, z.x + bias.x), r.x),
                                     fmaf(gate.y, activate(e.act, z.y + bias.y), r.y),
                                     fmaf(gate.z, activate(e.act, z.z + bias.z), r.z),
                                     fmaf(gate.w, activate(e.act, z.w + bias.w), r.w));
        if (!in_bounds(at + 3, M * N)) continue;
        if constexpr (kBf16Out)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(y) + at) =
                make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(y) + at) = o;
    }
}

// The weight-streaming path's reduce kernel (skinny_reduce_kernel) with the epilogue.  What the caller gave is loaded
// before the wait for the partials: the chain's first kernel, the activations' conversion, is a plain launch.
template <bool kBf16Out>
__global__ void __launch_bounds__(256) epilogue_reduce_kernel(const float* __restrict__ partial,
                                                              const int* __restrict__ rowexp, void* y, int M, int N,
                                                              int cpt, int64_t units, int P, int segmax,
                                                              int64_t partial_elems, const Epilogue e) {
    __shared__ int64_t seg_base[skinny::kMaxCtas];
    __shared__ int count;
    const int w = blockIdx.x;
    const int t = blockIdx.y * 2 + (threadIdx.x >> 7), r = threadIdx.x & 127;
    const int n = w * skinny::BW + r;
    const bool inside = t < M && n < N;
    const int64_t at = static_cast<int64_t>(t) * N + n;
    int seg = -1;
    float bias = 0.0f, gate = 1.0f, res = 0.0f;
    if (inside && in_bounds(at, static_cast<int64_t>(M) * N)) {
        seg = segment_of(e, t, M);
        bias = bias_of(e, N, n);
        if (e.residual != nullptr)
            res = kBf16Out ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[at])
                           : static_cast<const float*>(e.residual)[at];
        if (seg >= 0) gate = gate_of(e, seg, N, n);
    }
    if (threadIdx.x == 0) count = skinny::list_segments(w, cpt, units, P, segmax, seg_base);
    ptx::grid_dependency_wait();                       // partials come from the kernel before
    __syncthreads();
    if (!inside || seg < 0) return;
    float z = skinny::sum_segments(partial, partial_elems, seg_base, count, M, t, r);
    z = ldexpf(z, rowexp[t]) + bias;
    const float o = fmaf(gate, activate(e.act, z), res);
    if constexpr (kBf16Out)
        static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(o);
    else
        static_cast<float*>(y)[at] = o;
}

}  // namespace epi
}  // namespace ql
