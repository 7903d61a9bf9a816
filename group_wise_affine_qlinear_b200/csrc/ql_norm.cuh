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
// The operation moves each row once and does a dozen flops per element, so DRAM bounds it; a row therefore stays in
// registers from its load to its stores.  What it must not do is fetch and combine the five vectors (weights, gate,
// scale, shift) again for every row: that alone is 2.5 times the row's bytes from L1 and half of the instructions
// (4608 x 4608, bf16: 59 us with the vectors read per row, 46% of all issue slots busy; 43 us, 3.9 TB/s, with them held in
// registers, premultiplied, for as long as the segment stays the same; 33792 rows 223 us, 5.6 TB/s; with an fp32 residual
// and two fp32 partials 467 us, 6.0 TB/s).  Forms, with what each measured against the other (bf16, one call on cold
// caches, some 7 us of each being the call's start and end):
//   D <= kGroupMax          8, 16 or 32 lanes per row, no block barrier, the next row loaded ahead into registers.  33792
//                           rows against the other forms: 72 columns 16 us to 22, 128 18 to 23, 256 26 to 25, 384 46 to
//                           35, 512 47 to 37: it pays up to 256 columns.
//   longer rows, a few      a CTA per row, straight from global memory (latency: everything is loaded at once).  148 rows
//                           of 4608 against the ring: 10 us to 12; 296 rows 14 to 14; 592 rows 18 to 16; 1184 rows 29 to
//                           20; but of 16384 columns 1184 rows 61 to 78 (the ring has one CTA per SM there).
//   longer rows, many       persistent CTAs over consecutive rows with a ring of rows in shared memory, filled by bulk
//                           copies while earlier rows are reduced and written
// Rows too wide for two of them in an SM's shared memory take a CTA per row at any number; with four pieces per thread that
// form has 1024 threads of 64 registers, spills (up to 532 bytes, fp32 with partials) and loads a piece's partials one
// after the other: 4096 x 8192, fp32 with three partials 194 us, 3.8 TB/s; 2048 x 18432 with two 271 us, 2.5 TB/s.
#pragma once

#include "ql_ptx.cuh"

namespace ql {
namespace norm {

constexpr int kMaxD = 32768;          // 1024 threads x 4 vectors of 8
constexpr int kGroupMax = 512;        // 32 lanes x 2 vectors of 8 (see above: the second pays no longer)
constexpr int kGroupWarps = 4;        // warps per CTA of the group form

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
    float inv_d;               // 1 / D
};

// Rows are read once: keep them out of L1, which holds the vectors.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// Eight fp32 values as four pairs: the packed fp32 instructions (two IEEE operations each) halve the arithmetic's issue
// slots, which at 18 warps per SM were half of what this kernel waited for.
struct F8 {
    uint64_t p[4];
};
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t o;
    asm("mov.b64 %0, {%1, %2};" : "=l"(o) : "f"(lo), "f"(hi));
    return o;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(v));
    return o;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t o;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(o) : "l"(a), "l"(b), "l"(c));
    return o;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t o;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(o) : "l"(a), "l"(b));
    return o;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t o;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(o) : "l"(a), "l"(b));
    return o;
}
__device__ __forceinline__ F8 splat(float v) {
    const uint64_t q = pair_of(v, v);
    return {{q, q, q, q}};
}
__device__ __forceinline__ F8 mul(const F8& a, const F8& b) {
    return {{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1]), mul2(a.p[2], b.p[2]), mul2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ F8 add(const F8& a, const F8& b) {
    return {{add2(a.p[0], b.p[0]), add2(a.p[1], b.p[1]), add2(a.p[2], b.p[2]), add2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ F8 fma(const F8& a, const F8& b, const F8& c) {
    return {{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1]), fma2(a.p[2], b.p[2], c.p[2]),
             fma2(a.p[3], b.p[3], c.p[3])}};
}

__device__ __forceinline__ F8 unpack_bf16x8(const uint4 v) {
    return {{pair_of(bf16_lo(v.x), bf16_hi(v.x)), pair_of(bf16_lo(v.y), bf16_hi(v.y)),
             pair_of(bf16_lo(v.z), bf16_hi(v.z)), pair_of(bf16_lo(v.w), bf16_hi(v.w))}};
}
__device__ __forceinline__ uint32_t bf16_pair(uint64_t v) {
    const float2 f = halves(v);
    return pack_bf16x2(f.x, f.y);
}
__device__ __forceinline__ uint4 pack_bf16x8(const F8& f) {
    return make_uint4(bf16_pair(f.p[0]), bf16_pair(f.p[1]), bf16_pair(f.p[2]), bf16_pair(f.p[3]));
}
__device__ __forceinline__ F8 unpack_f32x8(const uint4 a, const uint4 b) {
    return {{pair_of(__uint_as_float(a.x), __uint_as_float(a.y)), pair_of(__uint_as_float(a.z), __uint_as_float(a.w)),
             pair_of(__uint_as_float(b.x), __uint_as_float(b.y)), pair_of(__uint_as_float(b.z), __uint_as_float(b.w))}};
}

// 8 elements of a parameter vector from element i on.
__device__ __forceinline__ F8 load_params(const void* p, int f32, int64_t i) {
    if (f32) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        return unpack_f32x8(__ldg(q), __ldg(q + 1));
    }
    return unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)));
}

// Sum of v over the CTA, through one shared float per warp, in a fixed order.  red: 32 floats, those past the CTA's
// warps zero.
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int nwarps = static_cast<int>(blockDim.x >> 5);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const float4* q = reinterpret_cast<const float4*>(red);
    float4 s = q[0];
    for (int i = 1; 4 * i < nwarps; ++i) {
        const float4 t = q[i];
        s = make_float4(s.x + t.x, s.y + t.y, s.z + t.z, s.w + t.w);
    }
    return (s.x + s.y) + (s.z + s.w);
}

template <int VPT>
__device__ __forceinline__ float sum_squares(const F8 (&v)[VPT]) {
    uint64_t a = 0, b = 0;                         // threads past the row's end hold zeros
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        a = fma2(v[j].p[0], v[j].p[0], a);
        b = fma2(v[j].p[1], v[j].p[1], b);
        a = fma2(v[j].p[2], v[j].p[2], a);
        b = fma2(v[j].p[3], v[j].p[3], b);
    }
    const float2 f = halves(add2(a, b));
    return f.x + f.y;
}

// The hardware's reciprocal root errs by two units at most, four of the roundings that the sum itself makes.
__device__ __forceinline__ float inv_rms(const Params& p, float ss) {
    return rsqrtf(fmaf(ss, p.inv_d, p.eps));
}

// A segment's vectors for one 8-element piece of the row: r = residual_scale x + v inv gain, h = r inv mod + shift.
struct Vectors {
    F8 gain, mod, shift;
};

// Starts the loads of a segment's vectors without waiting for them: load_vectors takes the vectors one by one (its
// registers are all but spoken for) and would wait for each.  One row of 4608: 5.3 -> 3.8 us.
template <bool kHasY, int VPT>
__device__ __forceinline__ void touch_vectors(const Params& p, int seg, int c0, int step) {
    const int64_t vec = static_cast<int64_t>(seg) * p.D;
    const int width = p.params_f32 ? 4 : 2;
    const auto touch = [&](const void* q, int64_t at) {
        if (q == nullptr) return;
        uint32_t unused;
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(unused) : "l"(static_cast<const uint8_t*>(q) + at * width));
    };
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = c0 + j * step;
        if (c >= p.D / 8) continue;
        if constexpr (kHasY) {
            touch(p.post_weight, 8 * c);
            touch(p.gate, vec + 8 * c);
        }
        touch(p.pre_weight, 8 * c);
        touch(p.scale, vec + 8 * c);
        touch(p.shift, vec + 8 * c);
    }
}

template <bool kHasY>
__device__ __forceinline__ void load_vectors(const Params& p, int seg, int c, Vectors& o) {
    const int64_t vec = static_cast<int64_t>(seg) * p.D;
    // every load before the first use; an absent vector is its neutral value
    const auto get = [&](const void* q, int64_t at, float none) {
        return q != nullptr ? load_params(q, p.params_f32, at + 8 * c) : splat(none);
    };
    F8 post, gate;
    if constexpr (kHasY) {
        post = get(p.post_weight, 0, 1.0f);
        gate = get(p.gate, vec, 1.0f);
    }
    const F8 pre = get(p.pre_weight, 0, 1.0f), scale = get(p.scale, vec, 0.0f);
    o.shift = get(p.shift, vec, 0.0f);
    if constexpr (kHasY) o.gain = mul(mul(splat(p.branch_scale), post), gate);
    o.mod = mul(add(splat(1.0f), scale), pre);
}

// r of one piece, from x (in r) and v, and its store at element `at`.
template <bool kXF32>
__device__ __forceinline__ void update(const Params& p, F8& r, const F8& v, float inv, const Vectors& w, int64_t at,
                                       bool store) {
    r = fma(mul(v, splat(inv)), w.gain, mul(splat(p.residual_scale), r));
    if (!store) return;
    if constexpr (kXF32) {
        ulonglong2* o = reinterpret_cast<ulonglong2*>(static_cast<float*>(p.r) + at);
        o[0] = make_ulonglong2(r.p[0], r.p[1]);
        o[1] = make_ulonglong2(r.p[2], r.p[3]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.r) + at) = pack_bf16x8(r);
    }
}

__device__ __forceinline__ void modulate(const Params& p, const F8& r, float inv, const Vectors& w, int64_t at,
                                         bool store) {
    const F8 o = fma(mul(r, splat(inv)), w.mod, w.shift);
    if (store) *reinterpret_cast<uint4*>(p.h + at) = pack_bf16x8(o);
}

// A row by a CTA, from the loaded x (in r) and v to its stores.  w: the vectors of the thread's pieces, or null to
// fetch them piece by piece.  row_done() runs once every thread has its inputs in registers: after the first
// reduction's barrier (a row without a reduction is the caller's to synchronize).  store(): whether to store, asked
// where the values are ready.
template <bool kXF32, bool kHasY, int VPT, class Store, class RowDone>
__device__ __forceinline__ void finish_row(const Params& p, F8 (&r)[VPT], const F8 (&v)[VPT], int64_t row,
                                           int seg, const Vectors* w, float (*red)[32], Store&& store, RowDone&& row_done) {
    const int nv = p.D / 8, tid = static_cast<int>(threadIdx.x), nthreads = static_cast<int>(blockDim.x);
    bool told = false;
    if constexpr (kHasY) {
        float inv = 1.0f;
        if (p.post_norm) {
            inv = inv_rms(p, row_sum(sum_squares<VPT>(v), red[0]));
            row_done();
            told = true;
        }
        const bool keep = store();
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid + j * nthreads;
            if (c >= nv) continue;
            Vectors t;
            if (w == nullptr) load_vectors<true>(p, seg, c, t);
            update<kXF32>(p, r[j], v[j], inv, w == nullptr ? t : w[j], row + 8 * c, keep);
        }
    }
    if (p.h != nullptr) {
        const float inv = inv_rms(p, row_sum(sum_squares<VPT>(r), red[1]));
        if (!told) row_done();
        told = true;
        const bool keep = store();
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = tid + j * nthreads;
            if (c >= nv) continue;
            Vectors t;
            if (w == nullptr) load_vectors<false>(p, seg, c, t);
            modulate(p, r[j], inv, w == nullptr ? t : w[j], row + 8 * c, keep);
        }
    }
    if (!told) row_done();
}

template <bool kF32>
struct Raw {                                       // 8 row elements as they lie in memory
    uint4 q[kF32 ? 2 : 1];
};
template <bool kF32>
__device__ __forceinline__ void fetch(const void* p, int64_t i, Raw<kF32>& o) {
    if constexpr (kF32) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        o.q[0] = ld_stream(q);
        o.q[1] = ld_stream(q + 1);
    } else {
        o.q[0] = ld_stream(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i));
    }
}
template <bool kF32>
__device__ __forceinline__ F8 unpack(const Raw<kF32>& o) {
    if constexpr (kF32) return unpack_f32x8(o.q[0], o.q[1]);
    else return unpack_bf16x8(o.q[0]);
}

// v plus the partials 1 .. S-1 of its 8 elements, added in order.
__device__ __forceinline__ F8 add_partials(const Params& p, int64_t at, F8 v) {
    for (int z = 1; z < p.S; ++z) {
        Raw<true> w;
        fetch<true>(p.y, static_cast<int64_t>(z) * p.M * p.D + at, w);
        v = add(v, unpack<true>(w));
    }
    return v;
}

// G = 8, 16 or 32 lanes per row; a warp takes `per_warp` rows (a multiple of 32 / G), 32 / G at a time.
template <bool kXF32, int kY, int VPT>
__global__ void __launch_bounds__(32 * kGroupWarps) norm_group_kernel(const Params p, int G, int64_t per_warp) {
    const int lane = static_cast<int>(threadIdx.x & 31), c0 = lane & (G - 1), nv = p.D / 8;
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * kGroupWarps + (threadIdx.x >> 5)) * per_warp;
    const int64_t end = min(first + per_warp, p.M);
    const int rows = 32 / G;
    if (first >= end) return;
    constexpr bool kYF = kY == kYF32;
    Raw<kXF32> xn[VPT];
    Raw<kYF> yn[VPT];
    Vectors w[VPT];
    int held = -1, next = -1;                      // segment of the held vectors; of the row loaded ahead (-1: skip)
    const auto load = [&](int64_t m) {
        next = -1;
        if (m >= end) return;
        next = p.seg != nullptr ? p.seg[m] : 0;
        if (next >= p.T) {
            if (c0 == 0) record_status(QL_ERR_INVALID_ARG);
            next = -1;
        }
        if (next < 0) return;                      // padding
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = c0 + j * G;
            if (c >= nv) continue;
            fetch<kXF32>(p.x, m * p.D + 8 * c, xn[j]);
            if constexpr (kY != kYNone) fetch<kYF>(p.y, m * p.D + 8 * c, yn[j]);
        }
    };
    const auto group_sum = [&](float v) {
        for (int o = G >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    };
    load(first + lane / G);
    for (int64_t base = first; base < end; base += rows) {
        const int64_t m = base + lane / G;
        const int seg = next;
        F8 r[VPT], v[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = c0 + j * G;
            r[j] = v[j] = splat(0.0f);
            if (seg < 0 || c >= nv) continue;
            r[j] = unpack<kXF32>(xn[j]);
            if constexpr (kY != kYNone) v[j] = unpack<kYF>(yn[j]);
            if constexpr (kYF) v[j] = add_partials(p, m * p.D + 8 * c, v[j]);
        }
        load(m + rows);
        if (seg >= 0 && seg != held) {
            held = seg;
            touch_vectors<kY != kYNone, VPT>(p, seg, c0, G);
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (c0 + j * G < nv) load_vectors<kY != kYNone>(p, seg, c0 + j * G, w[j]);
        }
        if constexpr (kY != kYNone) {
            float inv = 1.0f;
            if (p.post_norm) inv = inv_rms(p, group_sum(sum_squares<VPT>(v)));
#pragma unroll
            for (int j = 0; j < VPT; ++j)
                if (c0 + j * G < nv) update<kXF32>(p, r[j], v[j], inv, w[j], m * p.D + 8 * (c0 + j * G), seg >= 0);
        }
        if (p.h == nullptr) continue;
        const float inv = inv_rms(p, group_sum(sum_squares<VPT>(r)));
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (c0 + j * G < nv) modulate(p, r[j], inv, w[j], m * p.D + 8 * (c0 + j * G), seg >= 0);
    }
}

// A CTA per row; up to 1024 threads of VPT pieces.
template <bool kXF32, int kY, int VPT>
__global__ void __launch_bounds__(1024) norm_row_kernel(const Params p) {
    __shared__ __align__(16) float red[2][32];
    if (threadIdx.x < 64) red[threadIdx.x >> 5][threadIdx.x & 31] = 0.0f;
    const int tid = static_cast<int>(threadIdx.x), nthreads = static_cast<int>(blockDim.x);
    const int64_t m = blockIdx.x;
    const int nv = p.D / 8;
    const int64_t row = m * p.D;
    constexpr bool kYF = kY == kYF32;
    Raw<kXF32> xr[VPT];
    Raw<kYF> yr[VPT];
    const int seg = p.seg != nullptr ? p.seg[m] : 0;
    if (seg >= p.T) {
        if (tid == 0) record_status(QL_ERR_INVALID_ARG);
        return;
    }
    if (seg < 0) return;                           // padding
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = tid + j * nthreads;
        if (c >= nv) continue;
        fetch<kXF32>(p.x, row + 8 * c, xr[j]);
        if constexpr (kY != kYNone) fetch<kYF>(p.y, row + 8 * c, yr[j]);
    }
    touch_vectors<kY != kYNone, VPT>(p, seg, tid, nthreads);
    __syncthreads();                               // red is zeroed
    // with one piece per thread the vectors fit beside the row and their loads go out with the row's
    Vectors w[1];
    if (VPT == 1 && tid < nv) load_vectors<kY != kYNone>(p, seg, tid, w[0]);
    F8 r[VPT], v[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int c = tid + j * nthreads;
        r[j] = v[j] = splat(0.0f);
        if (c >= nv) continue;
        r[j] = unpack<kXF32>(xr[j]);
        if constexpr (kY != kYNone) v[j] = unpack<kYF>(yr[j]);
        if constexpr (kYF) v[j] = add_partials(p, row + 8 * c, v[j]);
    }
    finish_row<kXF32, kY != kYNone, VPT>(p, r, v, row, seg, VPT == 1 ? w : nullptr, red, [] { return true; }, [] {});
}

// Persistent CTAs: CTA b takes the rows [b M / B, (b + 1) M / B) of a grid of B; row i of its list lies in ring stage
// i % stages, as [x row | S rows of y].  Thread 0 issues a row's copies `stages` rows ahead, as soon as the stage's
// previous row is in registers; the row's segment is fetched one row earlier still and passed on in shared memory.  A
// padding row is not copied.  With one or two pieces per thread the segment's vectors are held in registers.
constexpr int kMaxStages = 4;
// Pieces per thread, most threads and CTAs per SM of the four configurations.
template <int kCfg> struct RingCfg;
template <> struct RingCfg<0> { static constexpr int kVpt = 1, kThreads = 256, kCtas = 3; };
template <> struct RingCfg<1> { static constexpr int kVpt = 2, kThreads = 320, kCtas = 2; };
template <> struct RingCfg<2> { static constexpr int kVpt = 2, kThreads = 512, kCtas = 1; };
template <> struct RingCfg<3> { static constexpr int kVpt = 4, kThreads = 512, kCtas = 1; };

__host__ __device__ constexpr uint32_t stage_bytes(int D, int x_bytes, int y_bytes, int S) {
    return static_cast<uint32_t>((D * x_bytes + 127) / 128 * 128 + S * ((D * y_bytes + 127) / 128 * 128));
}

template <bool kXF32, int kY, int kCfg>
__global__ void __launch_bounds__(RingCfg<kCfg>::kThreads, RingCfg<kCfg>::kCtas)
    norm_ring_kernel(const Params p, int stages) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(16) float red[2][32];
    __shared__ __align__(8) uint64_t full[kMaxStages];
    __shared__ int seg_s[kMaxStages];
    __shared__ int abort_flag;
    constexpr int VPT = RingCfg<kCfg>::kVpt;
    constexpr bool kHold = VPT <= 2;
    constexpr int kXB = kXF32 ? 4 : 2, kYB = kY == kYNone ? 0 : kY == kYF32 ? 4 : 2;
    const int tid = static_cast<int>(threadIdx.x), nthreads = static_cast<int>(blockDim.x);
    const int D = p.D, nv = D / 8;
    const int S = kY == kYNone ? 0 : kY == kYF32 ? p.S : 1;
    const uint32_t xb = static_cast<uint32_t>(D) * kXB, yb = static_cast<uint32_t>(D) * kYB;
    const uint32_t x_pad = (xb + 127) / 128 * 128, y_pad = (yb + 127) / 128 * 128;
    const uint32_t stage_size = x_pad + static_cast<uint32_t>(S) * y_pad;
    const int64_t m_end = p.M * (blockIdx.x + 1) / gridDim.x;
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) ptx::mbar_init(&full[i], 1);
        abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (tid < 64) red[tid >> 5][tid & 31] = 0.0f;
    __syncthreads();

    const auto segment = [&](int64_t m) { return p.seg != nullptr && m < m_end ? p.seg[m] : 0; };
    // thread 0: start row m's copies into a stage, or mark it as one to skip
    const auto issue = [&](int64_t m, int s, int seg) {
        if (m >= m_end) return;
        seg_s[s] = seg;
        if (stalled(kStallNorm)) return;                   // the checked build can hold every copy back
        if (seg < 0 || seg >= p.T) {
            ptx::mbar_arrive(&full[s]);
            return;
        }
        uint8_t* dst = ring + s * stage_size;
        ptx::mbar_arrive_expect_tx(&full[s], xb + S * yb);
        ptx::bulk_load(dst, static_cast<const uint8_t*>(p.x) + m * xb, xb, &full[s]);
        for (int z = 0; z < S; ++z)
            ptx::bulk_load(dst + x_pad + z * y_pad, static_cast<const uint8_t*>(p.y) + (z * p.M + m) * yb, yb, &full[s]);
    };
    int64_t m = p.M * blockIdx.x / gridDim.x;
    int next_seg = 0;                                      // of row m + stages, the next to copy
    if (tid == 0) {
        test_delay(kDelayActivations);                     // the checked build can hold the copies back (qlinear_test_delay)
        int segs[kMaxStages];                              // all of them at once: their loads are the start's latency
#pragma unroll
        for (int i = 0; i < kMaxStages; ++i) segs[i] = segment(m + i);
#pragma unroll
        for (int i = 0; i < kMaxStages; ++i)
            if (i < stages) issue(m + i, i, segs[i]);
        next_seg = segment(m + stages);
    }
    Vectors w[kHold ? VPT : 1];
    int held = -1;
    const auto hold = [&](int seg) {
        held = seg;
        touch_vectors<kY != kYNone, VPT>(p, seg, tid, nthreads);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (tid + j * nthreads < nv) load_vectors<kY != kYNone>(p, seg, tid + j * nthreads, w[kHold ? j : 0]);
    };
    if (kHold) {                                           // the first row's vectors, while it is on its way
        const int seg = segment(m);
        if (seg >= 0 && seg < p.T) hold(seg);
    }
    // a wait of some thread has expired: no more stores or copies, the same barriers
    const auto aborted = [&] { return *const_cast<volatile int*>(&abort_flag) != 0; };
    test_delay(kDelayEpilogue);                            // (and the warps)
    int s = 0;
    uint32_t phase = 0;
    for (; m < m_end; ++m) {
        ptx::mbar_wait(&full[s], phase, &abort_flag);
        const int seg = seg_s[s];
        const auto refill = [&] {
            if (tid == 0 && !aborted()) {
                issue(m + stages, s, next_seg);
                next_seg = segment(m + stages + 1);
            }
        };
        if (seg < 0 || seg >= p.T) {                                   // the same in every thread
            if (tid == 0 && seg >= p.T) record_status(QL_ERR_INVALID_ARG);
            __syncthreads();                                           // every thread has read seg_s[s]
            refill();
        } else {
            if (kHold && seg != held) hold(seg);
            const uint8_t* src = ring + s * stage_size;
            F8 r[VPT], v[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int c = tid + j * nthreads;
                r[j] = v[j] = splat(0.0f);
                if (c >= nv) continue;
                const uint4* q = reinterpret_cast<const uint4*>(src + 8 * kXB * c);
                if constexpr (kXF32) r[j] = unpack_f32x8(q[0], q[1]);
                else r[j] = unpack_bf16x8(q[0]);
                if constexpr (kY == kYBf16) v[j] = unpack_bf16x8(*reinterpret_cast<const uint4*>(src + x_pad + 16 * c));
                if constexpr (kY == kYF32) {
                    for (int z = 0; z < S; ++z) {
                        const uint4* y = reinterpret_cast<const uint4*>(src + x_pad + z * y_pad + 32 * c);
                        const F8 f = unpack_f32x8(y[0], y[1]);
                        v[j] = z == 0 ? f : add(v[j], f);
                    }
                }
            }
            const int reductions = (kY != kYNone && p.post_norm ? 1 : 0) + (p.h != nullptr ? 1 : 0);
            if (reductions == 0) __syncthreads();                      // no barrier would tell that the stage is read
            finish_row<kXF32, kY != kYNone, VPT>(p, r, v, m * D, seg, kHold ? w : nullptr, red, [&] { return !aborted(); }, refill);
            // with two reductions a row each one's buffer is read before the other's barrier; with one, the next row
            // must not overtake its readers
            if (reductions == 1) __syncthreads();
        }
        if (++s == stages) {
            s = 0;
            phase ^= 1u;
        }
    }
    if (tid == 0 && aborted()) {
        // no copy may land after the CTA: wait for the phase that each barrier is in (the limit also bounds the wait for
        // one with no copy under way)
        for (int i = 0; i < stages; ++i)
            ptx::mbar_wait(&full[i], ptx::mbar_test(ptx::smem_addr(&full[i]), 0) ? 1u : 0u, nullptr);
    }
}

}  // namespace norm
}  // namespace ql
