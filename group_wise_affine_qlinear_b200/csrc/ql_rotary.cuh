// Norms of queries and keys for each head, with the rotation by positions of several axes in the same pass.
//
//   n[m][h][d] = x[m][h][d] / sqrt(mean_d x[m][h][d]^2 + eps) * weight[d]            (optional)
//   the first 2 P elements of a head are P pairs (a, b): elements i and i + P, or 2 i and 2 i + 1;
//   pair i turns by the angle 2 pi turns[i] pos[axes[i]][m]:  (a, b) <- (a cos - b sin, b cos + a sin)
//
// All of it in fp32, but the angle: position times turns is formed in 64 bits and its whole turns are dropped before it
// is rounded (at position 2^20 a product in 32 bits is off by up to a sixteenth of a turn's radian).  Rounded once.
//
// A head is some hundred bytes to a kilobyte that is read and written once, so DRAM bounds it.  G lanes hold a head in
// registers from load to store, each two pieces of 8 elements that hold 8 pairs; the sines and cosines of a token
// depend on the lane alone and stay in registers over the heads.
#pragma once

#include "ql_norm.cuh"

namespace ql {
namespace rotary {

constexpr int kMaxD = 512;             // 32 lanes x 16 elements
constexpr int kWarps = 4;

struct Heads {
    const void* in;
    void* out;
    int64_t in_token, in_head, out_token, out_head;    // strides in elements
    const void* weight;                                // [D] or null (1)
    int heads;
};

struct Params {
    Heads set[2];              // queries; keys (heads 0: none)
    const void* pos;           // [A][M]
    const double* turns;       // [P] turns per unit of position
    const int* axes;           // [P]
    const int* seg;            // [M] or null
    int64_t M;
    int D, P, A;
    int pos_type;              // ql_pos_type
    int norm;
    int weight_f32;
    int parts;                 // warps that share a token's heads
    float eps, inv_d;
};

__device__ __forceinline__ double position(const Params& p, int axis, int64_t m) {
    const int64_t i = axis * p.M + m;
    if (p.pos_type == QL_POS_I32) return static_cast<double>(__ldg(static_cast<const int*>(p.pos) + i));
    if (p.pos_type == QL_POS_I64) return static_cast<double>(__ldg(static_cast<const long long*>(p.pos) + i));
    return static_cast<double>(__ldg(static_cast<const float*>(p.pos) + i));
}

// A token's heads (or its part of them) per warp, 32 / G heads at a time.  kAdjacent: pairs (2 i, 2 i + 1).
template <bool kF32, bool kAdjacent, int G>
__global__ void __launch_bounds__(32 * kWarps) heads_kernel(const Params p) {
    using norm::Raw;
    constexpr int kPer = 32 / G;                       // heads at a time
    constexpr int kOwn = 8 / kPer;                     // angles a lane computes; the others' come by shuffles
    const int lane = static_cast<int>(threadIdx.x & 31), slot = lane & (G - 1), which = lane / G;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t m = unit / p.parts;
    const int part = static_cast<int>(unit - m * p.parts);
    if (m >= p.M || (p.seg != nullptr && __ldg(p.seg + m) < 0)) return;

    // the lane's two pieces of 8 elements: 8 pairs of the turned part, or what is left behind it
    const bool turned = slot < p.P / 8;
    const int ea = kAdjacent || !turned ? 16 * slot : 8 * slot;
    const int eb = turned && !kAdjacent ? ea + p.P : ea + 8;
    const bool has_a = ea < p.D && slot * 16 < p.D, has_b = has_a && eb < p.D;

    float c[8], s[8];
    {
        float oc[kOwn], os[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int pair = 8 * slot + which * kOwn + i;
            oc[i] = 1.0f;
            os[i] = 0.0f;
            if (turned) {
                const int axis = __ldg(p.axes + pair);
                if (static_cast<unsigned>(axis) < static_cast<unsigned>(p.A)) {
                    double t = position(p, axis, m) * __ldg(p.turns + pair);
                    t -= rint(t);
                    sincospif(2.0f * static_cast<float>(t), &os[i], &oc[i]);
                } else {
                    record_status(QL_ERR_INVALID_ARG);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = __shfl_sync(0xFFFFFFFFu, oc[i % kOwn], (i / kOwn) * G + slot);
            s[i] = __shfl_sync(0xFFFFFFFFu, os[i % kOwn], (i / kOwn) * G + slot);
        }
    }

    const int first[2] = {0, (p.set[0].heads + kPer - 1) / kPer};
    const int groups = first[1] + (p.set[1].heads + kPer - 1) / kPer;
    const int g0 = static_cast<int>(static_cast<int64_t>(part) * groups / p.parts);
    const int g1 = static_cast<int>(static_cast<int64_t>(part + 1) * groups / p.parts);
    for (int k = 0; k < 2; ++k) {
        const Heads& hs = p.set[k];
        const int lo = max(g0, first[k]), hi = k == 0 ? min(g1, first[1]) : g1;
        if (lo >= hi) continue;
        norm::F8 wa = norm::splat(1.0f), wb = wa;
        if (p.norm && hs.weight != nullptr) {
            if (has_a) wa = norm::load_params(hs.weight, p.weight_f32, ea);
            if (has_b) wb = norm::load_params(hs.weight, p.weight_f32, eb);
        }
        for (int g = lo; g < hi; ++g) {
            const int h = (g - first[k]) * kPer + which;
            const bool live = h < hs.heads;
            norm::F8 a = norm::splat(0.0f), b = a;
            const int64_t at = m * hs.in_token + h * hs.in_head;
            Raw<kF32> ra, rb;
            if (live && has_a) {
                norm::fetch<kF32>(hs.in, at + ea, ra);
                if (has_b) norm::fetch<kF32>(hs.in, at + eb, rb);
                a = norm::unpack<kF32>(ra);
                if (has_b) b = norm::unpack<kF32>(rb);
            }
            if (p.norm) {
                const norm::F8 v[2] = {a, b};
                float ss = norm::sum_squares<2>(v);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                const norm::F8 inv = norm::splat(rsqrtf(fmaf(ss, p.inv_d, p.eps)));
                a = norm::mul(norm::mul(a, inv), wa);
                b = norm::mul(norm::mul(b, inv), wb);
            }
            if (turned) {
                float fa[8], fb[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = norm::halves(a.p[i]), v = norm::halves(b.p[i]);
                    fa[2 * i] = u.x;
                    fa[2 * i + 1] = u.y;
                    fb[2 * i] = v.x;
                    fb[2 * i + 1] = v.y;
                }
                if constexpr (kAdjacent) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a.p[i] = norm::pair_of(fa[2 * i] * c[i] - fa[2 * i + 1] * s[i], fa[2 * i + 1] * c[i] + fa[2 * i] * s[i]);
                        b.p[i] = norm::pair_of(fb[2 * i] * c[4 + i] - fb[2 * i + 1] * s[4 + i],
                                               fb[2 * i + 1] * c[4 + i] + fb[2 * i] * s[4 + i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        a.p[i] = norm::pair_of(fa[2 * i] * c[2 * i] - fb[2 * i] * s[2 * i],
                                               fa[2 * i + 1] * c[2 * i + 1] - fb[2 * i + 1] * s[2 * i + 1]);
                        b.p[i] = norm::pair_of(fb[2 * i] * c[2 * i] + fa[2 * i] * s[2 * i],
                                               fb[2 * i + 1] * c[2 * i + 1] + fa[2 * i + 1] * s[2 * i + 1]);
                    }
                }
            }
            if (live && has_a) {
                const int64_t to = m * hs.out_token + h * hs.out_head;
                const auto store = [&](const norm::F8& v, int64_t i) {
                    if constexpr (kF32) {
                        ulonglong2* q = reinterpret_cast<ulonglong2*>(static_cast<float*>(hs.out) + i);
                        q[0] = make_ulonglong2(v.p[0], v.p[1]);
                        q[1] = make_ulonglong2(v.p[2], v.p[3]);
                    } else {
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(hs.out) + i) = norm::pack_bf16x8(v);
                    }
                };
                store(a, to + ea);
                if (has_b) store(b, to + eb);
            }
        }
    }
}

}  // namespace rotary
}  // namespace ql
