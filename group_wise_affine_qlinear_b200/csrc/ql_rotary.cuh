// Norms of queries and keys for each head, with the rotation by positions of several axes in the same pass.
//
//   n[m][h][d] = x[m][h][d] / sqrt(mean_d x[m][h][d]^2 + eps) * weight[d]            (optional)
//   the first 2 P elements of a head are P pairs (a, b): elements i and i + P, or 2 i and 2 i + 1;
//   pair i turns by the angle 2 pi turns[i] pos[axes[i]][m]:  (a, b) <- (a cos - b sin, b cos + a sin)
//
// All of it in fp32, but the angle: position times turns is formed in 64 bits and its whole turns are dropped before it
// is rounded (at position 2^20 a product in 32 bits is off by up to 0.06 rad).  Rounded once.
//
// A head is some hundred bytes to a kilobyte that is read and written once, so DRAM bounds many tokens: 33792 of 24 heads
// of 256, written by heads, 134 us, 6.2 TB/s; 32760 of 24 of 128, neighbours paired, 67 us, 6.0 TB/s; 4608 of 36 of 256
// 41 us, 4.1 TB/s (4608 warps on 2960 places).  G lanes hold a head in registers from ring to store, each two pieces of 8
// elements that hold 8 pairs; weights and angles of a lane are folded into four vectors per token, so an element costs two
// packed operations and the norm's factor.  (Against it, the two 2048^2 canvases above: one load at a time 199 us, loads a
// group ahead in registers 174, selects around the ring's copies 140; persistent warps over runs of tokens 225, persistent
// CTAs that share a token's angles 275, two to nine warps per token 186 to 349: DRAM wants neighbouring tokens at the same
// time, and a unit's start is not free.  4608 tokens: two warps per token 44, three 46.)
#pragma once

#include "ql_norm.cuh"

namespace ql {
namespace rotary {

constexpr int kMaxD = 512;             // 32 lanes x 16 elements
constexpr int kWarps = 4;
constexpr int kStages = 4;             // (3: the two canvases above 142 us, the video clip 71; 4: 136, 69; 6: 140, 71; 8: 144, 83)

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
    int at_once_log;           // log2 of the heads of a token that a warp holds at a time
    float eps, inv_d;
};

// Elements from a set's first to one past its last, as it lies in memory.
__device__ __forceinline__ int64_t span(const Params& p, int64_t token, int64_t head, int heads) {
    return (p.M - 1) * token + (heads - 1) * head + p.D;
}
// Whether 8 elements from `at` on lie within the set that starts at `base`.
template <int kSize>
__device__ __forceinline__ bool piece_in(const uint8_t* at, const void* base, int64_t span) {
    const int64_t first = (at - static_cast<const uint8_t*>(base)) / kSize;
    return in_bounds(first, span) && in_bounds(first + 7, span);
}

__device__ __forceinline__ double position(const Params& p, int64_t i) {
    if (p.pos_type == QL_POS_I32) return static_cast<double>(__ldg(static_cast<const int*>(p.pos) + i));
    if (p.pos_type == QL_POS_I64) return static_cast<double>(__ldg(static_cast<const long long*>(p.pos) + i));
    return static_cast<double>(__ldg(static_cast<const float*>(p.pos) + i));
}

__device__ __forceinline__ float rsqrt_fast(float v) {  // 2 units; a subnormal counts as zero
    float o;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(o) : "f"(v));
    return o;
}
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
    const float2 f = norm::halves(v);
    return norm::pair_of(f.y, f.x);
}

// A warp holds 32 / G heads at a time: `at_once` of each of its 32 / G / at_once tokens, whose heads (or, for few tokens,
// a part of them) it walks.  kAdjacent: pairs (2 i, 2 i + 1).  kFull: D = 16 G, every lane has both of its pieces.
template <bool kF32, bool kAdjacent, int G, bool kFull>
__global__ void __launch_bounds__(32 * kWarps, kF32 ? 4 : 5) heads_kernel(const Params p) {
    using norm::F8;
    __shared__ uint4 ring[kWarps][kStages][kF32 ? 4 : 2][32];
    __shared__ __align__(16) float kept[kWarps][2][32][8];     // cosines and sines of a token's pairs, G slots of 8 per token
    constexpr int kPer = 32 / G;
    constexpr int kSize = kF32 ? 4 : 2;
    const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5), slot = lane & (G - 1);
    const int at_once = 1 << p.at_once_log, which = (lane / G) & (at_once - 1), token = lane / G >> p.at_once_log;
    int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    int part = 0;
    if (p.parts > 1) {
        part = static_cast<int>(unit % p.parts);
        unit /= p.parts;
    }
    int64_t m = unit * (kPer >> p.at_once_log) + token;
    const bool live = m < p.M && (p.seg == nullptr || __ldg(p.seg + m) >= 0);
    if (!__any_sync(0xFFFFFFFFu, live)) return;
    if (!live) m = 0;                                  // (its heads are neither read nor written)

    // the lane's two pieces of 8 elements: 8 pairs of the turned part, or what is left behind it
    const bool turned = slot < p.P / 8;
    const int ea = kAdjacent || !turned ? 16 * slot : 8 * slot;
    const int eb = turned && !kAdjacent ? ea + p.P : ea + 8;
    const bool has_a = kFull || 16 * slot < p.D, has_b = kFull || (has_a && eb < p.D);

    // the warp's groups of at_once heads: [lo, hi) of the queries', then of the keys'
    const int nq = (p.set[0].heads + at_once - 1) >> p.at_once_log;
    const int groups = nq + ((p.set[1].heads + at_once - 1) >> p.at_once_log);
    int g0 = 0, g1 = groups;
    if (p.parts > 1) {
        g0 = static_cast<int>(static_cast<int64_t>(part) * groups / p.parts);
        g1 = static_cast<int>(static_cast<int64_t>(part + 1) * groups / p.parts);
    }
    const auto head_in = [&](int set, int g) {
        const Heads& hs = p.set[set];
        return static_cast<const uint8_t*>(hs.in) +
               (m * hs.in_token + static_cast<int64_t>(g * at_once + which) * hs.in_head + ea) * kSize;
    };
    const auto heads_from = [&](int set, int g) {      // > 0: the lane has one
        return live ? p.set[set].heads - g * at_once - which : 0;
    };
    // The groups pass through a ring in shared memory, every lane copying and reading its own pieces: kStages - 1 of them
    // are on their way at any time, the first while the angles are formed.
    // (Lanes past a head's end or the last head copy nothing.  The two vectors of 8 fp32, and the two pieces of 16
    // neighbours, share their 32-byte sectors: those copies go through L1, so that a sector is fetched once.)
    constexpr bool kThroughL1 = kF32 || kAdjacent;
    int fset = g0 < nq ? 0 : 1, fstage = 0, fend = fset ? g1 : min(g1, nq), fg = g0;       // what is copied next
    int fleft = heads_from(fset, g0 - fset * nq);
    int64_t fstep = p.set[fset].in_head * (at_once * kSize);
    const uint8_t* from = head_in(fset, g0 - fset * nq);
    const auto fetch = [&] {
        if (fg < fend) {
            uint4 (*to)[32] = ring[warp][fstage];
            const Heads& hs = p.set[fg < nq ? 0 : 1];
            const int64_t all = span(p, hs.in_token, hs.in_head, hs.heads);
#pragma unroll
            for (int v = 0; v < (kF32 ? 2 : 1); ++v) {
                if (fleft > 0 && has_a && piece_in<kSize>(from, hs.in, all))
                    ptx::copy16_async_of<kThroughL1>(&to[v][lane], from + 16 * v);
                if (fleft > 0 && has_b && piece_in<kSize>(from + (eb - ea) * kSize, hs.in, all))
                    ptx::copy16_async_of<kThroughL1>(&to[(kF32 ? 2 : 1) + v][lane], from + (eb - ea) * kSize + 16 * v);
            }
            fleft -= at_once;
            from += fstep;
            if (++fg == nq && fg < g1) {
                fend = g1;
                fleft = heads_from(1, 0);
                fstep = p.set[1].in_head * (at_once * kSize);
                from = head_in(1, 0);
            }
        }
        fstage = (fstage + 1) % kStages;
        ptx::copy_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch();

    // a token's angles, shared by the lanes of its at_once heads
    float (*const cosines)[8] = kept[warp][0] + token * G;
    float (*const sines)[8] = kept[warp][1] + token * G;
    if (turned) {
        for (int i = which; i < 8; i += at_once) {
            float c = 1.0f, s = 0.0f;
            const int axis = in_bounds(8 * slot + i, p.P) ? __ldg(p.axes + 8 * slot + i) : -1;
            if (static_cast<unsigned>(axis) < static_cast<unsigned>(p.A)) {
                const int64_t at = axis * p.M + m;
                double t = in_bounds(at, p.A * p.M) ? position(p, at) * __ldg(p.turns + 8 * slot + i) : 0.0;
                t -= rint(t);
                sincospif(2.0f * static_cast<float>(t), &s, &c);
            } else {
                record_status(QL_ERR_INVALID_ARG);
            }
            cosines[slot][i] = c;
            sines[slot][i] = s;
        }
    }
    __syncwarp();
    int stage = 0;

    for (int set = 0; set < 2; ++set) {
        const Heads& hs = p.set[set];
        const int lo = set == 0 ? g0 : max(g0 - nq, 0), hi = set == 0 ? min(g1, nq) : g1 - nq;
        if (lo >= hi) continue;
        // Weights and angles in one: with (a, b) a lane's pieces, their outputs are a ca + b sa and b cb + a sb; neighbours
        // are pairs within a piece, there x (cos, cos) + swapped x (-sin, sin), and the weights of the swapped x swapped.
        F8 ca = norm::splat(1.0f), cb = ca, sa, sb;
        if (p.norm && hs.weight != nullptr) {
            if (has_a && in_bounds(ea + 7, p.D)) ca = norm::load_params(hs.weight, p.weight_f32, ea);
            if (has_b && in_bounds(eb + 7, p.D)) cb = norm::load_params(hs.weight, p.weight_f32, eb);
        }
        if (turned) {
            float c[8], s[8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                *reinterpret_cast<float4*>(c + 4 * i) = *reinterpret_cast<const float4*>(&cosines[slot][4 * i]);
                *reinterpret_cast<float4*>(s + 4 * i) = *reinterpret_cast<const float4*>(&sines[slot][4 * i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kAdjacent) {
                    sa.p[i] = norm::mul2(swapped(ca.p[i]), norm::pair_of(-s[i], s[i]));
                    sb.p[i] = norm::mul2(swapped(cb.p[i]), norm::pair_of(-s[4 + i], s[4 + i]));
                    ca.p[i] = norm::mul2(ca.p[i], norm::pair_of(c[i], c[i]));
                    cb.p[i] = norm::mul2(cb.p[i], norm::pair_of(c[4 + i], c[4 + i]));
                } else {
                    const uint64_t cc = norm::pair_of(c[2 * i], c[2 * i + 1]);
                    sa.p[i] = norm::mul2(cb.p[i], norm::pair_of(-s[2 * i], -s[2 * i + 1]));
                    sb.p[i] = norm::mul2(ca.p[i], norm::pair_of(s[2 * i], s[2 * i + 1]));
                    ca.p[i] = norm::mul2(ca.p[i], cc);
                    cb.p[i] = norm::mul2(cb.p[i], cc);
                }
            }
        }
        uint8_t* to = static_cast<uint8_t*>(hs.out) +
                      (m * hs.out_token + static_cast<int64_t>(lo * at_once + which) * hs.out_head + ea) * kSize;
        const int64_t out_step = hs.out_head * (at_once * kSize);
        int left = heads_from(set, lo);
        for (int g = lo; g < hi; ++g, left -= at_once, to += out_step) {
            fetch();                                   // into what was read a group ago
            ptx::copy_async_wait<kStages - 1>();
            norm::Raw<kF32> ra, rb;
#pragma unroll
            for (int v = 0; v < (kF32 ? 2 : 1); ++v) {
                ra.q[v] = ring[warp][stage][v][lane];
                rb.q[v] = ring[warp][stage][(kF32 ? 2 : 1) + v][lane];
            }
            stage = (stage + 1) % kStages;
            F8 a = norm::unpack<kF32>(ra), b = norm::unpack<kF32>(rb);
            if (!has_a) a = norm::splat(0.0f);         // (for the sum of squares)
            if (!has_b) b = norm::splat(0.0f);
            F8 inv;
            if (p.norm) {
                const F8 v[2] = {a, b};
                float ss = norm::sum_squares<2>(v);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                inv = norm::splat(rsqrt_fast(fmaf(ss, p.inv_d, p.eps)));
            }
            F8 ya, yb;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ya.p[i] = norm::mul2(a.p[i], ca.p[i]);
                yb.p[i] = norm::mul2(b.p[i], cb.p[i]);
                if (turned) {
                    ya.p[i] = norm::fma2(kAdjacent ? swapped(a.p[i]) : b.p[i], sa.p[i], ya.p[i]);
                    yb.p[i] = norm::fma2(kAdjacent ? swapped(b.p[i]) : a.p[i], sb.p[i], yb.p[i]);
                }
                if (p.norm) {
                    ya.p[i] = norm::mul2(ya.p[i], inv.p[i]);
                    yb.p[i] = norm::mul2(yb.p[i], inv.p[i]);
                }
            }
            const auto store = [&](const F8& v, uint8_t* q) {
                if constexpr (kF32) {
                    reinterpret_cast<ulonglong2*>(q)[0] = make_ulonglong2(v.p[0], v.p[1]);
                    reinterpret_cast<ulonglong2*>(q)[1] = make_ulonglong2(v.p[2], v.p[3]);
                } else {
                    *reinterpret_cast<uint4*>(q) = norm::pack_bf16x8(v);
                }
            };
            const int64_t all = span(p, hs.out_token, hs.out_head, hs.heads);
            if (left > 0 && has_a && piece_in<kSize>(to, hs.out, all)) store(ya, to);
            if (left > 0 && has_b && piece_in<kSize>(to + (eb - ea) * kSize, hs.out, all)) store(yb, to + (eb - ea) * kSize);
        }
    }
    ptx::copy_async_wait<0>();
}

}  // namespace rotary
}  // namespace ql
