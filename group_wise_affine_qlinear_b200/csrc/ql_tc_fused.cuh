// Fused-dequant tensor-core GEMM for large M (tcgen05, TMEM operands and accumulators).
//
// y[m][n] = rowscale[m] * sum_k xh[m][k] * wh(n, k)
//   xh    f16 activations prescaled per row by a power of two (prepass)
//   wh    RN_f16(s * q + b): the affine grid of aimarketly "Ideogram-4-IQ4_M",
//         "What IQ4 means here", formed by one fused f16x2 multiply-add from the
//         exact code q, i.e. rounded once; q is a 4-bit code, or an 8-bit code of
//         the Q8 pack (huggingface "SceneWorks/ideogram-4-mlx", Versions) with the
//         same per-64 scale and bias
// Operands are f16 (A and B must share a type in kind::f16); the accumulator is
// fp32 in tensor memory.  One K-step is exactly one 64-wide quantization group,
// so every weight row needs one (scale, bias) pair per step.
//
// The MMA computes the transposed tile D[n][m] = sum_k wh(n, k) xh(m, k), for
// two groups of 128 weight rows that share one activation tile:
//   A = dequantized weights, 128 rows x 64 k per group, written by the
//       dequantizers straight into tensor memory (tcgen05.st), never into
//       shared memory;
//   B = activations, 192 tokens x 64 k, TMA-loaded into shared memory with the
//       128-byte swizzle, read by both groups' MMAs;
//   D = per group 128 lanes (weight rows) x 192 columns (tokens), fp32.
// Keeping the dequantized tiles out of shared memory leaves shared memory to the
// activation stream, and serving 256 weight rows from each activation tile
// halves the L2 -> SM traffic per FLOP compared with one group.  TMEM holds the
// two accumulators (2 x 192 columns) and two A stages of 2 x 32 columns: all
// 512 columns, so each accumulator is single-buffered; the MMA of the next tile
// waits only for its own group to be drained, which overlaps half the epilogue.
//
// Warp roles of one persistent CTA per SM (640 threads):
//   warps 0-7   dequantizers: warp w owns TMEM lanes 32*(w%4).. of group w/4,
//               one weight row per thread, every K-step
//   warp 8      TMA producer of activation tiles
//   warps 9, 11 single-thread MMA issuers for groups 0 / 1 (warp 9 also allocates TMEM);
//               (one thread issuing for both groups measured slower)
//   warp 10     TMA producer of code and parameter tiles
//   warps 12-19 epilogue: all eight drain group 0, then group 1 (warp w takes TMEM
//               lanes 32*(w%4).. and half of the tokens): TMEM -> registers ->
//               rowscale -> bf16/fp32 -> a 32x32 staging block in shared memory ->
//               TMA tensor store (which also clips the ragged edges of y)
// Rings: X (activation tiles, one K-step each, freed by MMA completion), C (codes +
// parameters of kS consecutive K-steps, freed once the dequantizers have read the
// last of them), A (TMEM weight stages, one K-step each); accumulators are freed per
// group by the epilogue.  Each MMA warp waits on one barrier and commits once per
// K-step: x_full[s] completes when the step's activation tile has landed and the
// dequantizers have written its TMEM stage, and the commit to x_empty[s] frees both
// the x stage and that step's A stage.  Issuing one tcgen05.mma costs its thread
// about 50 cycles, against 96 tensor cycles for a 128 x 192 x 16 MMA, so the
// issuers are held back by the tensor pipe, not by issue.  What the kernel loses
// against the pipe's peak is the time a step is not ready (its weights, its
// activations, a drained accumulator) and the clock that the board's power cap
// leaves while the tensor core and the dequantizers run together.
//
// SwiGLU mode (kSwiGLU): the DiT block's MLP is a SwiGLU of three Linears (jimmysue
// "Ideogram 4" notes, sec. 2.1 and 2.8); this mode fuses the gate and up
// projections and the gating.  A tile's two row groups are the same 128 rows of
// the gate weight (group 0) and of the up weight (group 1), loaded as two
// 128-row code boxes from two tensor maps, with their (scale, bias) pairs
// interleaved the same way by the parameter prepass.  The two accumulators then
// hold g and u for the same 128 intermediate columns and 192 tokens, and each of
// the 8 epilogue warps reads both for its lane quarter and half of the tokens and
// writes h = silu(g) * u = g / (1 + e^-g) * u in fp32 (the exponential and the
// division through the SFU's exp2 and reciprocal), rounded once.
//
// Adapter mode (kLora): y += sum_j t[m][j] B[a][n][j] for the low-rank adapter a of every row m, t = s x . A^T (an
// earlier kernel).  The product is more K for the same accumulators: after the G quantization groups the unit that
// owns the end of K runs extra K-steps whose weight operand is B itself (bf16, bit for bit) and whose activation
// operand is t, scaled like the row's activations and cut into two bf16, t = hi + lo to 2^-16 relative (the MMA's
// type is per instruction: these steps run in bf16, whose exponents cannot overflow where f16's could).  A "part" is 8
// columns of B under 16 of t's, [hi 8 | lo 8]; a tile's distinct adapters lie side by side, r / 8 parts each (in
// SwiGLU mode the gate's r / 8, then the up's, each multiplied for its own row group alone), four parts to a step; a
// token's row is zero outside its own adapter's parts.  So a tile pays for the adapters in it (one step per 32 / r of them),
// nothing travels through memory a second time, and y is rounded once.  B comes by TMA through the code ring (a code
// stage per extra step), t by TMA too, eight rows at a time, but for the eights that meet several adapters.
//
// Epilogue mode (kAct): y = residual + gate[seg] * act(acc + bias), on the accumulator's way out (epilogue_role).
#pragma once

#include "ql_ptx.cuh"
#include "ql_dequant_f16.cuh"
#include "ql_epilogue.cuh"

namespace ql {
namespace fused {

constexpr int BWG = 128;                // weight rows per group (MMA M, TMEM lanes)
constexpr int NG = 2;                   // groups per tile
constexpr int BW = NG * BWG;            // weight rows per tile
constexpr int BT = 192;                 // tokens per tile (MMA N, TMEM columns)
constexpr int BK = 64;
constexpr int UK = 16;
constexpr int kDequantWarps = 8;
constexpr int kWarpTmaX = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpTmaC = 10;
constexpr int kWarpMma2 = 11;
constexpr int kWarpEpi0 = 12;           // 12..19: quarters 0..3 of group 0, then of group 1
constexpr int kEpiWarps = 4 * NG;
constexpr int kThreads = (kWarpEpi0 + kEpiWarps) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAccCol = 0;         // accumulator of group g at columns [g*BT, (g+1)*BT)
constexpr uint32_t kAStageCol = NG * BT;// A stage s, group g at columns [384 + 64 s + 32 g, +32)
constexpr int NA = 2;                   // TMEM weight stages
static_assert(kAStageCol + NA * NG * 32 <= kTmemCols, "tensor memory budget");

constexpr uint32_t kXBytes = BT * BK * 2;   // 24 KB
constexpr uint32_t kCodeRowBytes = 128;     // code bytes of one weight row per code stage

// NX activation stages; NC code stages, each holding kS = 128 / (8 * B) consecutive K-steps of B-bit
// codes (128 bytes of every one of the tile's 256 rows, stored with the 128-byte swizzle: 4 steps of
// 4-bit codes, 2 of 8-bit codes) with their (scale, bias) pairs; epilogue staging blocks of 32 x 32
// outputs of OB bytes each (2: bf16, 4: fp32), NB of them per epilogue warp.  Wide code rows keep the
// number of rows the TMA unit fetches per K-step low (64 rows of 128 bytes instead of 256 of 32); the
// narrower bf16 staging leaves room for a fifth activation stage.
template <int NX, int NC, int B, int OB, int NB>
struct Cfg {
    static constexpr int kNX = NX, kNC = NC, kBits = B, kOutBytes = OB, kNB = NB;
    static constexpr int kS = kCodeRowBytes / (BK * B / 8);
    static constexpr uint32_t kCBytes = BW * kCodeRowBytes;
    static constexpr uint32_t kPBytes = BW * 4 * kS;
    static constexpr uint32_t kStageBytes = 32 * 32 * OB;
    static constexpr uint32_t kEpiBytes = kEpiWarps * NB * kStageBytes;
    static constexpr uint32_t kOffX = 0;
    static constexpr uint32_t kOffC = kOffX + NX * kXBytes;
    static constexpr uint32_t kOffP = kOffC + NC * kCBytes;
    static constexpr uint32_t kOffEpi = kOffP + NC * kPBytes;
    static constexpr uint32_t kOffBar = kOffEpi + kEpiBytes;
    static constexpr uint32_t kNumBars = 2 * NX + 2 * NC + 1 + NG + NG;
    // the A stage of K-step i is released by the x_empty phase of step i - NA, which must not complete
    // its next phase (step i - NA + NX) before the dequantizers have written step i
    static_assert(NX >= NA, "the activation ring is at least as deep as the TMEM weight ring");
    static constexpr uint32_t kOffMisc = kOffBar + kNumBars * 8;
    static constexpr uint32_t kSmemBytes = kOffMisc + 16 + 1024;   // + alignment slack
    static_assert(kXBytes % 1024 == 0 && kCBytes % 1024 == 0, "swizzle atoms need 1 KB alignment");
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// The configuration of each (code width, output type): bf16 outputs stage in half the space of fp32
// ones (split-K partials, fp32 outputs), which keep one staging block per warp to stay in budget.
template <int B, bool kBf16Out>
struct PickCfg;
template <> struct PickCfg<4, true> { using type = Cfg<5, 2, 4, 2, 2>; };
template <> struct PickCfg<4, false> { using type = Cfg<4, 2, 4, 4, 1>; };
template <> struct PickCfg<8, true> { using type = Cfg<5, 2, 8, 2, 2>; };
template <> struct PickCfg<8, false> { using type = Cfg<4, 2, 8, 4, 1>; };
// Epilogue mode: two staging blocks per warp, one worked on while the next one's residual arrives, and two buffers of a
// tile's vectors (row scales of 96 tokens, bias and gate of 2 x 32 columns); they take the room of an activation stage.
constexpr uint32_t kEpiVectorBytes = BT / 2 * 4 + 2 * NG * 32 * 4;
template <class Base>
struct EpiCfg : Base {
    static_assert(Base::kNB == 2, "two staging blocks");
    static constexpr uint32_t kOffVec = Base::kOffMisc + 16;
    static constexpr uint32_t kSmemBytes = Base::kSmemBytes + kEpiWarps * 2 * kEpiVectorBytes;
    static_assert(kOffVec % 8 == 0 && kSmemBytes <= 232448, "shared memory budget");
};
template <int B, bool kBf16Out>
struct PickEpiCfg;
template <int B> struct PickEpiCfg<B, true> { using type = EpiCfg<Cfg<4, 2, B, 2, 2>>; };
template <int B> struct PickEpiCfg<B, false> { using type = EpiCfg<Cfg<3, 2, B, 4, 2>>; };

struct Params {
    float* rowscale;      // [M] 2^e_m
    void* y;              // [M][N] bf16 or fp32
    int M, N, G;
    int num_t, num_w;     // token tiles, weight tiles
    int splits;           // K slices per tile (split-K instantiations; 1 otherwise)
};

// Adapter mode: the operands of the extra K-steps.
struct LoraParams : Params {
    CUtensorMap map_b[2];        // B of the layer (of gate and up) as (r, N, L), boxes of part_cols(r8) columns
    CUtensorMap map_tw;          // tw as [M][16 parts], boxes of 64 columns x 8 rows
    const __nv_bfloat16* tw;     // [M][parts][hi 8 | lo 8]: t 2^-e_m, zeros for a row without an adapter
    const int* row_slot;         // [M] place of the row's adapter in its token tile's list, or -1
    const int* tile_count;       // [num_t] distinct adapters of the token tile
    const int* tile_list;        // [num_t][BT]
    int r8;                      // r / 8
    int parts;                   // parts per adapter: r8, in SwiGLU mode 2 r8
};
// Columns of a box of B: an extra step needs at most four parts of an adapter.
__host__ __device__ constexpr int part_cols(int r8) { return r8 < 4 ? 8 * r8 : 32; }
struct EpiParams : Params {
    epi::Epilogue e;
};
template <bool kLora, bool kEpi> struct PickParams { using type = Params; };
template <> struct PickParams<true, false> { using type = LoraParams; };
template <> struct PickParams<false, true> { using type = EpiParams; };

__device__ __forceinline__ void tile_coords(int t, int num_w, int& t_blk, int& w_blk) {
    // weight tiles fastest: a wave of CTAs shares one or two activation row blocks
    // (streamed from HBM once) and sweeps the whole (L2-resident) packed weight.
    t_blk = t / num_w;
    w_blk = t - t_blk * num_w;
}

// Position in a ring of N stages for the i-th use overall.
template <int N>
__device__ __forceinline__ void ring_pos(uint32_t i, int& stage, uint32_t& phase) {
    stage = static_cast<int>(i % N);
    phase = (i / N) & 1u;
}

// Two f32 as two bf16 pairs with hi + lo = v to 2^-16 relative: hi is v cut to bf16, lo the rest rounded.  A
// non-finite v stays in hi (lo 0), so it reaches the outputs of its own row as itself.
__device__ __forceinline__ uint32_t bf16_part(float v0, float v1, bool lo) {
    const uint32_t u0 = __float_as_uint(v0), u1 = __float_as_uint(v1);
    const bool f0 = (u0 & 0x7F800000u) != 0x7F800000u, f1 = (u1 & 0x7F800000u) != 0x7F800000u;
    const float h0 = f0 ? __uint_as_float(u0 & 0xFFFF0000u) : v0, h1 = f1 ? __uint_as_float(u1 & 0xFFFF0000u) : v1;
    return lo ? pack_bf16x2(f0 ? v0 - h0 : 0.0f, f1 ? v1 - h1 : 0.0f) : pack_bf16x2(h0, h1);
}

constexpr int kNoEpilogue = -1;     // kAct of a plain layer; else a ql_activation

// Registers per thread in epilogue mode: its warps take what the TMA and MMA warps (one warpgroup) do not need.
constexpr int kEpiRegs = 120, kIssueRegs = 48, kLaunchRegs = 96;
static_assert(kDequantWarps * kLaunchRegs + 4 * kIssueRegs + kEpiWarps * kEpiRegs <= (kThreads / 32) * kLaunchRegs,
              "the warps' shares fit what the block is launched with");
template <bool kEpi>
__device__ __forceinline__ bool give_registers() {
    if constexpr (kEpi) ptx::fewer_registers<kIssueRegs>();
    return true;
}

// The epilogue warps of the epilogue mode.  Warp (quarter, half) drains its lanes of group 0, then of group 1, in chunks of
// 32 tokens x 32 columns, as in the plain epilogue; chunk q of its run passes through staging block q % 2, to which the
// residual of its tokens is copied while chunk q - 1 is worked on, and from which its outputs go to y, 16 bytes a lane.
// Lane l works on columns 8 i + l / 4 (i < 4) and, for j < 4, on tokens 8 j + 2 (l % 4) and + 1 of a chunk: the fragment of
// the accumulator that transposing matrix stores (and loads, for the residual) take to a token's row, eight elements an
// instruction.  A row's 16-byte pieces are permuted by its number, so that neither matrices nor rows meet in a bank.
//
// The drain is not hidden: tensor memory holds one accumulator per group, and the next tile's products wait for it.  A chunk
// takes a warp 1100 cycles, 1450 with a residual; 4608 x 4608 x 4608 137 us (the plain epilogue 135), with gate and residual
// 143, silu 147, gelu_tanh 150, gelu 151 (their two special functions a value are a tile's 3 us).  With two K-steps a tile
// takes 6.5 us: 3.6 its six chunks per warp, 1.2 the K-steps (0.55 to 0.6 each up to eight), the rest the hand-over between
// products and drain; 4608 x 128 x 4608 has three such tiles one behind the other, and 6.7 us of launches and start.
// What cost most before: registers.  At the launch's 96 a thread the compiler spilled values on their way from memory and
// waited for each (146 us whatever else was done).  One 16-bit store per element instead of matrix stores 147 and, with gelu,
// 184; outputs and residual through the TMA, whose rows are 64 bytes here, 145 and 150 with a residual.  No gain: storing a
// chunk while the next is read, announcing the groups' accumulators apart, two values sharing a reciprocal.
template <bool kBf16Out, int kAct>
__device__ __forceinline__ void epilogue_role(const EpiParams& p, uint32_t stage0, uint32_t stage_bytes, uint32_t vec0,
                                              uint32_t tmem_base,
                                              uint64_t* acc_full, uint64_t* acc_empty, volatile int* abort_flag, int quarter,
                                              int half, int lane) {
    constexpr int kHalf = BT / 32 / 2, kPast = -2, kElem = kBf16Out ? 2 : 4;
    constexpr int kPieces = 32 * kElem / 16, kRows = 32 / kPieces;     // a copy: kPieces lanes per row, kRows rows at a time
    const int lt = 2 * (lane & 3), ln = lane >> 2;
    const uint32_t mat_off = 64u * (lane & 7) + 16u * ((lane >> 3) ^ ((lane >> 1) & 3));                // bf16
    const int row0 = lane / kPieces, piece = lane % kPieces;
    // (the copies' rows row0 + kRows k differ in a multiple of 8 or 4: one permutation or two for all of them)
    const auto piece_at = [&](int k) {
        const int row = row0 + kRows * k;
        return static_cast<uint32_t>(row * 32 * kElem + 16 * (piece ^ (kBf16Out ? (row >> 1) & 3 : row & 7)));
    };
    const int num_tiles = p.num_t * p.num_w, N = p.N;
    const bool has_res = p.e.residual != nullptr;
    const int64_t row_step = static_cast<int64_t>(N) * kElem;
    const uint32_t acc = tmem_base + kAccCol + static_cast<uint32_t>(32 * kHalf * half) + (static_cast<uint32_t>(quarter * 32) << 16);
    const int m_off = 32 * kHalf * half, n_off = quarter * 32;         // this warp's part of a tile

    // the residual of 32 tokens from m on and 32 columns from n on
    const auto copy_residual = [&](uint32_t block, int m, int n) {
        const int left = p.M - m - row0, col = n + piece * (16 / kElem);
        const uint8_t* from = static_cast<const uint8_t*>(p.e.residual) + (m + row0) * row_step + static_cast<int64_t>(col) * kElem;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const bool in = kRows * k < left && col < N &&
                            in_bounds(static_cast<int64_t>(m + row0 + kRows * k) * N + col + 16 / kElem - 1,
                                      static_cast<int64_t>(p.M) * N);
            ptx::copy16_async(stage0 + block * stage_bytes + piece_at(k), in ? from + kRows * k * row_step : p.e.residual, in);
        }
    };
    // What a tile needs beside its accumulators is copied, asynchronously too, while the tile before is drained: its row
    // scales, and both groups' bias and gate (as they are; the gate of the tile's first token), in one of two buffers.
    // (Fetched into registers they cost more of them than there are, and the loads' latency with the spills.)
    constexpr uint32_t kRsAt = 0, kBiasAt = 32 * kHalf * 4, kGateAt = kBiasAt + NG * 128;
    static_assert(kGateAt + NG * 128 == kEpiVectorBytes, "the buffers' size");
    const bool wide = p.e.params_f32 != 0;
    const auto copy_rows = [&](uint32_t to, int t_blk) {
#pragma unroll
        for (int c = 0; c < kHalf; ++c) {
            const int m = t_blk * BT + m_off + 32 * c + lane;
            const int at = min(m, p.M - 1);
            if (in_bounds(at, p.M)) ptx::copy4_async(to + kRsAt + 128u * c + 4u * lane, p.rowscale + at);
        }
    };
    const auto copy_vector = [&](uint32_t to, const void* from, int rows, int row, int n) {    // 32 columns from n on
        if (from == nullptr) return;
        const int col = wide ? n + lane : n + 2 * (lane & 15);                         // (those past N are not stored)
        const int64_t at = static_cast<int64_t>(row) * N + (col < N ? col : 0);
        if (!in_bounds(at + (wide ? 0 : 1), static_cast<int64_t>(rows) * N)) return;
        ptx::copy4_async(to + (wide ? 4u * lane : 4u * (lane & 15)), static_cast<const uint8_t*>(from) + (wide ? 4 * at : 2 * at));
    };
    const auto vector_at = [&](const void* given, uint32_t at, float none) {           // of the lane's columns
        float4 o = make_float4(none, none, none, none);
        if (given != nullptr) {
            if (wide)
                o = make_float4(ptx::ld_shared_f32(at + 4u * ln), ptx::ld_shared_f32(at + 4u * ln + 32u),
                                ptx::ld_shared_f32(at + 4u * ln + 64u), ptx::ld_shared_f32(at + 4u * ln + 96u));
            else
                o = make_float4(ptx::ld_shared_bf16(at + 2u * ln), ptx::ld_shared_bf16(at + 2u * ln + 16u),
                                ptx::ld_shared_bf16(at + 2u * ln + 32u), ptx::ld_shared_bf16(at + 2u * ln + 48u));
        }
        return o;
    };
    // Segment of token 32 c + lane of a tile; kPast beyond M.  Without a gate all segments are alike: a chunk's tokens would
    // go in one round per segment otherwise, and a zero's sign would depend on its neighbours' (4608 x 4608 x 4608 with bias
    // and four segments in no order 167 us a call, so 152 as without ids).
    const auto segment = [&](int t_blk, int c) {
        const int m = t_blk * BT + m_off + 32 * c + lane;
        const int s = m < p.M ? epi::segment_of(p.e, m, p.M) : kPast;
        return p.e.gate == nullptr ? min(s, 0) : s;
    };

    ptx::grid_dependency_wait();                       // the row scales come from the kernels before this one
    int t_blk, w_blk, seg[kHalf];
    tile_coords(blockIdx.x, p.num_w, t_blk, w_blk);
#pragma unroll
    for (int c = 0; c < kHalf; ++c) seg[c] = segment(t_blk, c);
    int held = max(__shfl_sync(0xFFFFFFFFu, seg[0], 0), 0);            // segment of the gate at hand
    copy_rows(vec0, t_blk);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        copy_vector(vec0 + kBiasAt + 128u * g, p.e.bias, 1, 0, w_blk * BW + g * BWG + n_off);
        copy_vector(vec0 + kGateAt + 128u * g, p.e.gate, p.e.T, held, w_blk * BW + g * BWG + n_off);
    }
    if (has_res) copy_residual(0, t_blk * BT + m_off, w_blk * BW + n_off);
    ptx::copy_async_commit();
    uint32_t block = 0, phase = 0;
    for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, phase ^= 1u) {
        int t_next, w_next;
        tile_coords(t, p.num_w, t_blk, w_blk);
        tile_coords(t + static_cast<int>(gridDim.x), p.num_w, t_next, w_next);     // (past the last tile: rows past M)
        const int m0 = t_blk * BT + m_off, tile_seg = held;
        const uint32_t vec = vec0 + phase * kEpiVectorBytes, vec_next = vec0 + (phase ^ 1u) * kEpiVectorBytes;
        uint32_t live[kHalf], uniform = 0;             // live tokens; bit c: chunk c's are all of segment tile_seg
#pragma unroll
        for (int c = 0; c < kHalf; ++c) {
            live[c] = __ballot_sync(0xFFFFFFFFu, seg[c] >= 0);
            if (__all_sync(0xFFFFFFFFu, seg[c] < 0 || seg[c] == tile_seg)) uniform |= 1u << c;
        }
        if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(acc_full, phase, abort_flag))) break;
        ptx::tc_fence_after_sync();
        uint32_t v[2][16];                             // a chunk's values: TMEM lanes 16 h .. + 15 of the warp's 32
        ptx::tmem_ld_16x256b_x4(acc, v[0]);
        ptx::tmem_ld_16x256b_x4(acc + (16u << 16), v[1]);
#pragma unroll 1
        for (int g = 0; g < NG; ++g) {
            const int n0 = w_blk * BW + g * BWG + n_off;
            uint8_t* y = static_cast<uint8_t*>(p.y) + (m0 + row0) * row_step +
                         (n0 + piece * (16 / kElem)) * static_cast<int64_t>(kElem);
            const bool col_in = n0 + piece * (16 / kElem) < N;
            float4 bias, gate;
#pragma unroll
            for (int c = 0; c < kHalf; ++c, block ^= 1u) {
                const uint32_t stage = stage0 + block * stage_bytes;
                const bool last = c + 1 == kHalf;
                // the next chunk's residual (the other block was read before the last __syncwarp), the next tile's rows
                if (has_res) {
                    if (!last) copy_residual(block ^ 1u, m0 + 32 * (c + 1), n0);
                    else if (g == 0) copy_residual(block ^ 1u, m0, n0 + BWG);
                    else copy_residual(block ^ 1u, t_next * BT + m_off, w_next * BW + n_off);
                }
                if (g == 1 && c == 0) {
                    copy_rows(vec_next, t_next);
#pragma unroll
                    for (int i = 0; i < kHalf; ++i) seg[i] = segment(t_next, i);
                }
                if (g == 1 && last) {
                    held = max(__shfl_sync(0xFFFFFFFFu, seg[0], 0), 0);
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        copy_vector(vec_next + kBiasAt + 128u * i, p.e.bias, 1, 0, w_next * BW + i * BWG + n_off);
                        copy_vector(vec_next + kGateAt + 128u * i, p.e.gate, p.e.T, held, w_next * BW + i * BWG + n_off);
                    }
                }
                ptx::copy_async_commit();
                ptx::tmem_wait_ld();
                if (last) {                            // the group's last values are in registers: its MMAs may go on
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&acc_empty[g]);
                }
                ptx::copy_async_wait<1>();             // all copies but the ones just begun
                __syncwarp();
                if (c == 0) {
                    bias = vector_at(p.e.bias, vec + kBiasAt + 128u * g, 0.0f);
                    gate = vector_at(p.e.gate, vec + kGateAt + 128u * g, 1.0f);
                }
                const float b4[4] = {bias.x, bias.y, bias.z, bias.w};
                // act(acc * row scale + bias), in place
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 rs = ptx::ld_shared_f32x2(vec + kRsAt + 128u * c + 32u * j + 4u * lt);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t* a = &v[i >> 1][4 * j + 2 * (i & 1)];
                        const float2 o = epi::activate_as<kAct>(fmaf(__uint_as_float(a[0]), rs.x, b4[i]),
                                                                fmaf(__uint_as_float(a[1]), rs.y, b4[i]));
                        a[0] = __float_as_uint(o.x);
                        a[1] = __float_as_uint(o.y);
                    }
                }
                // residual + gate * act into the block; kRes: it holds the residual; kAll: for every token, else for
                // those in `mask`, the others keep what the block holds
                const auto finish = [&](auto res, auto all, uint32_t mask, const float4 w) {
                    constexpr bool kRes = decltype(res)::value, kAll = decltype(all)::value;
                    const float w4[4] = {w.x, w.y, w.z, w.w};
                    uint32_t b[4][4] = {};
                    if constexpr (kRes && kBf16Out) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) ptx::ldmatrix_x4_trans(stage + 512 * j + mat_off, b[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in0 = kAll || ((mask >> (8 * j + lt)) & 1u) != 0;
                        const bool in1 = kAll || ((mask >> (8 * j + lt + 1)) & 1u) != 0;
                        if constexpr (kBf16Out) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t* a = &v[i >> 1][4 * j + 2 * (i & 1)];
                                const float o0 = bf16_lo(b[j][i]), o1 = bf16_hi(b[j][i]);
                                const float y0 = kRes ? fmaf(w4[i], __uint_as_float(a[0]), o0) : w4[i] * __uint_as_float(a[0]);
                                const float y1 = kRes ? fmaf(w4[i], __uint_as_float(a[1]), o1) : w4[i] * __uint_as_float(a[1]);
                                b[j][i] = pack_bf16x2(in0 ? y0 : o0, in1 ? y1 : o1);
                            }
                            ptx::stmatrix_x4_trans(stage + 512 * j + mat_off, b[j]);
                        } else {
                            uint32_t at[8];
                            float r[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int token = lt + (i & 1);
                                at[i] = stage + 1024u * j + 128u * token + 4u * (ln & 3) + 16u * ((2u * (i >> 1) + (ln >> 2)) ^ token);
                                r[i] = kRes ? ptx::ld_shared_f32(at[i]) : 0.0f;
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float y = fmaf(w4[i >> 1], __uint_as_float(v[i >> 2][4 * j + (i & 3)]), r[i]);
                                ptx::st_shared_f32(at[i], ((i & 1) ? in1 : in0) ? y : r[i]);
                            }
                        }
                    }
                };
                if ((uniform >> c) & 1u) {
                    if (has_res) finish(std::true_type{}, std::true_type{}, 0u, gate);
                    else finish(std::false_type{}, std::true_type{}, 0u, gate);
                } else {                               // one round per segment among the chunk's tokens
                    if (!has_res) {
#pragma unroll
                        for (int k = 0; k < kPieces; ++k) ptx::st_shared_zero16(stage + piece_at(k));
                        __syncwarp();
                    }
                    const int seg_c = segment(t_blk, c);
                    for (uint32_t todo = live[c]; todo != 0;) {
                        const int s = __shfl_sync(0xFFFFFFFFu, seg_c, __ffs(todo) - 1);
                        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, seg_c == s);
                        todo &= ~mask;
                        float w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[i] = epi::gate_of(p.e, s, N, min(n0 + ln + 8 * i, N - 1));
                        finish(std::true_type{}, std::false_type{}, mask, make_float4(w[0], w[1], w[2], w[3]));
                        __syncwarp();                  // the next round reads what other lanes wrote
                    }
                }
                if (!last || g == 0) {
                    const uint32_t next = acc + (last ? static_cast<uint32_t>(BT) : g * static_cast<uint32_t>(BT) + 32u * (c + 1));
                    ptx::tmem_ld_16x256b_x4(next, v[0]);
                    ptx::tmem_ld_16x256b_x4(next + (16u << 16), v[1]);
                }
                __syncwarp();
                const uint32_t rows = col_in ? live[c] >> row0 : 0u;
                uint4 o[4];
#pragma unroll
                for (int k0 = 0; k0 < kPieces; k0 += 4) {              // four rows' loads, then their stores
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] = ptx::ld_shared_v4(stage + piece_at(k0 + k));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (((rows >> (kRows * (k0 + k))) & 1u) != 0 &&
                            in_bounds((m0 + row0 + 32 * c + kRows * (k0 + k)) * static_cast<int64_t>(N) + n0 +
                                          (piece + 1) * (16 / kElem) - 1, static_cast<int64_t>(p.M) * N))
                            *reinterpret_cast<uint4*>(y + (32 * c + kRows * (k0 + k)) * row_step) = o[k];
                }
                __syncwarp();                          // the block may be filled again
            }
        }
    }
    ptx::copy_async_wait<0>();                         // no copy lands after the CTA's end
}

// map_codes2: the up weight's codes in SwiGLU mode (128-row boxes, like map_codes there); unused otherwise.
// kSplitK: every tile's K-steps are cut into p.splits slices, each its own work unit; a unit writes the
// fp32 partial of its slice through map_y, a 3-D map over partials [splits][M][N], and a separate
// reduction sums the slices in order (for shapes with fewer tiles than SMs).
template <bool kBf16Out, class C, bool kSwiGLU = false, bool kSplitK = false, bool kLora = false, int kAct = kNoEpilogue>
__global__ void __launch_bounds__(kThreads, 1) fused_gemm_kernel(
    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_codes,
    const __grid_constant__ CUtensorMap map_codes2, const __grid_constant__ CUtensorMap map_params,
    const __grid_constant__ CUtensorMap map_y, const __grid_constant__ typename PickParams<kLora, kAct != kNoEpilogue>::type p) {
    constexpr bool kEpi = kAct != kNoEpilogue;
    constexpr int NX = C::kNX, NC = C::kNC;
    static_assert(!kSwiGLU || C::kBits == 4, "the SwiGLU pair is built for 4-bit codes");
    static_assert(!kSplitK || (!kSwiGLU && !kBf16Out), "split-K units write fp32 partials of a plain layer");
    static_assert(!kEpi || (!kSwiGLU && !kSplitK && !kLora), "the epilogue mode is a plain layer's");
    static_assert(kBf16Out == (C::kOutBytes == 2), "the staging blocks are sized for the output type");
    constexpr int kCodeWords = BK * C::kBits / 32;      // 32-bit code words of one row per K-step
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* x_full = bars;
    uint64_t* x_empty = x_full + NX;
    uint64_t* c_full = x_empty + NX;
    uint64_t* c_empty = c_full + NC;
    uint64_t* acc_full = c_empty + NC;          // one per tile
    uint64_t* acc_empty = acc_full + 1;         // one per group
    uint64_t* drain = acc_empty + NG;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int num_tiles = p.num_t * p.num_w;
    // Work units: a tile, or with kSplitK a (K slice, tile) pair, slice-major so that a wave of CTAs still
    // shares activation row blocks.  Unit u covers the K-steps [kb0, kb1) of tile t.
    const int num_units = kSplitK ? num_tiles * p.splits : num_tiles;
    auto unit = [&](int u, int& t, int& kb0, int& kb1) {
        if constexpr (kSplitK) {
            const int z = u / num_tiles;
            t = u - z * num_tiles;
            kb0 = static_cast<int>((static_cast<int64_t>(z) * p.G) / p.splits);
            kb1 = static_cast<int>((static_cast<int64_t>(z + 1) * p.G) / p.splits);
        } else {
            t = u;
            kb0 = 0;
            kb1 = p.G;
        }
    };
    // Adapter mode: the extra K-steps of unit u are the parts [p0, p1) of its token tile, four to a step.  A tile's
    // slices share them out like the groups of K.
    auto lora_parts = [&](int u, int t_blk, int& p0, int& p1) {
        p0 = p1 = 0;
        if constexpr (kLora) {
            p1 = p.tile_count[t_blk] * p.parts;
            if constexpr (kSplitK) {
                const int z = u / num_tiles, steps = (p1 + 3) / 4;
                p0 = 4 * static_cast<int>((static_cast<int64_t>(z) * steps) / p.splits);
                p1 = min(p1, 4 * static_cast<int>((static_cast<int64_t>(z + 1) * steps) / p.splits));
            }
        }
    };
    // Every role walks the same units in the same order: the X and A ring positions follow the K-step
    // count, the C ring position the code-stage count (a unit's steps in stages of kS, the last partial).

    if (threadIdx.x == 0) {
        // a K-step's x stage is released by both MMA warps' commits, which also release its A stage
        // x_full[s]: the step's activation tile has landed (the producer's expect_tx and the TMA) and its
        // TMEM weight stage is written (one arrival per dequantizer warp), so the MMA warps wait once
        for (int i = 0; i < NX; ++i) { ptx::mbar_init(&x_full[i], 1 + kDequantWarps); ptx::mbar_init(&x_empty[i], NG); }
        for (int i = 0; i < NC; ++i) { ptx::mbar_init(&c_full[i], 1); ptx::mbar_init(&c_empty[i], kDequantWarps); }
        ptx::mbar_init(&acc_full[0], NG);
        static_assert(kWarpEpi0 % 4 == 0, "epilogue warp w must own TMEM lane quarter w % 4");
        // an accumulator is drained by all 8 epilogue warps (a lane quarter and half of the tokens each)
        for (int g = 0; g < NG; ++g) ptx::mbar_init(&acc_empty[g], kEpiWarps);
        for (int g = 0; g < NG; ++g) ptx::mbar_init(drain + g, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kWarpTmaX && lane == 0) ptx::prefetch_tensormap(&map_x);
    if (warp == kWarpEpi0 && lane == 0) ptx::prefetch_tensormap(&map_y);
    if (warp == kWarpTmaC && lane == 0) {
        ptx::prefetch_tensormap(&map_codes);
        if constexpr (kSwiGLU) ptx::prefetch_tensormap(&map_codes2);
        ptx::prefetch_tensormap(&map_params);
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(tmem_slot, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;

    if (warp < kDequantWarps) {
        // ---------------------------------------------------------------- dequantizers
        test_delay(kDelayDequant);   // the checked build can hold this role back (qlinear_test_delay)
        const int grp = warp >> 2;                 // weight-row group
        const int quarter = warp & 3;              // TMEM lanes 32*quarter .. +31
        const int r = grp * BWG + quarter * 32 + lane;   // weight row within the tile
        const int sw = r & 7;                      // the 128-byte swizzle of row r's 16-byte pieces
        const uint8_t* crow0 = smem + C::kOffC + r * kCodeRowBytes;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        uint32_t i = 0, ci = 0;                    // K-step and code-stage counters
        bool ok = true;
        for (int un = blockIdx.x; un < num_units && ok; un += gridDim.x) {
            int t, kb0, kb1;
            unit(un, t, kb0, kb1);
            for (int kc = kb0; kc < kb1 && ok; kc += C::kS, ++ci) {
                int cs;
                uint32_t cph;
                ring_pos<NC>(ci, cs, cph);
                // Codes arrive far ahead of the tensor core: unpack them into registers first
                // and wait for the TMEM stage only when the result is ready to be written.
                if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&c_full[cs], cph, abort_flag))) { ok = false; break; }
                const uint8_t* crow = crow0 + cs * C::kCBytes;
                const uint32_t* sbs = reinterpret_cast<const uint32_t*>(smem + C::kOffP + cs * C::kPBytes);
                const int nsteps = min(C::kS, kb1 - kc);
                for (int st = 0; st < nsteps; ++st, ++i) {
                    const int as = static_cast<int>(i % NA);
                    uint32_t a[32];
                    const uint32_t sb = sbs[st * BW + r];
                    const __half2 sb2 = half2_of(sb);
                    const __half2 s2 = __low2half2(sb2);
                    const __half2 b2 = __high2half2(sb2);
                    if constexpr (C::kBits == 4) {
                        // step st is pieces 2st, 2st+1 of the row (16 codes each)
                        const uint4 c0 = *reinterpret_cast<const uint4*>(crow + (((2 * st) ^ sw) << 4));
                        const uint4 c1 = *reinterpret_cast<const uint4*>(crow + (((2 * st + 1) ^ sw) << 4));
                        if (st + 1 == nsteps) {            // the stage's codes and parameters are in registers
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(&c_empty[cs]);
                        }
                        const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
                        for (int c = 0; c < 8; ++c) dequant_word(words[c], s2, b2, &a[4 * c]);
                    } else {
                        // step st is pieces 4st .. 4st+3 of the row (16 byte codes each)
                        uint4 cv[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            cv[c] = *reinterpret_cast<const uint4*>(crow + (((4 * st + c) ^ sw) << 4));
                        if (st + 1 == nsteps) {
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(&c_empty[cs]);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            dequant_word8(cv[c].x, s2, b2, &a[8 * c + 0]);
                            dequant_word8(cv[c].y, s2, b2, &a[8 * c + 2]);
                            dequant_word8(cv[c].z, s2, b2, &a[8 * c + 4]);
                            dequant_word8(cv[c].w, s2, b2, &a[8 * c + 6]);
                        }
                    }
                    // TMEM stage `as` was last read by the MMAs of K-step i - NA: their commit completes
                    // that step's x_empty phase (one commit per MMA warp releases both stages)
                    if (i >= static_cast<uint32_t>(NA)) {
                        int xs;
                        uint32_t xph;
                        ring_pos<NX>(i - NA, xs, xph);
                        if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&x_empty[xs], xph, abort_flag))) {
                            ok = false;
                            break;
                        }
                    }
                    ptx::tc_fence_after_sync();
                    ptx::tmem_st_32x32b_x32(tmem_base + lane_addr + kAStageCol + 64u * as + 32u * grp, a);
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&x_full[i % NX]);   // TMEM stage of step i written
                }
            }
            if constexpr (kLora) {
                // extra K-steps: a code stage holds the step's boxes of B, one per adapter (and projection) that the
                // step meets, each [256 rows][cols]; a thread's row gives 8 columns per part, twice (under hi and lo)
                ptx::grid_dependency_wait();               // the tiles' adapter lists come from an earlier kernel
                int t_blk, w_blk;
                tile_coords(t, p.num_w, t_blk, w_blk);
                int p0, p1;
                lora_parts(un, t_blk, p0, p1);
                const int cols = part_cols(p.r8);
                const bool inside = (kSwiGLU ? w_blk * BWG + quarter * 32 + lane : w_blk * BW + r) < p.N;
                for (; p0 < p1 && ok; p0 += 4, ++i, ++ci) {
                    int cs;
                    uint32_t cph;
                    ring_pos<NC>(ci, cs, cph);
                    if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&c_full[cs], cph, abort_flag))) { ok = false; break; }
                    const uint8_t* box = smem + C::kOffC + cs * C::kCBytes + r * cols * 2;
                    int seg = p0 / p.r8, part = p0 - seg * p.r8, skip = part;
                    uint32_t a[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (inside && p0 + c < p1 && (!kSwiGLU || (seg & 1) == grp)) {
                            v = *reinterpret_cast<const uint4*>(box + 16 * (part - skip));
                            v.x = finite_bf16x2(v.x);
                            v.y = finite_bf16x2(v.y);
                            v.z = finite_bf16x2(v.z);
                            v.w = finite_bf16x2(v.w);
                        }
                        a[8 * c] = a[8 * c + 4] = v.x;
                        a[8 * c + 1] = a[8 * c + 5] = v.y;
                        a[8 * c + 2] = a[8 * c + 6] = v.z;
                        a[8 * c + 3] = a[8 * c + 7] = v.w;
                        if (++part == p.r8) {              // on to the next adapter's box
                            part = skip = 0;
                            ++seg;
                            box += BW * cols * 2;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&c_empty[cs]);
                    if (i >= static_cast<uint32_t>(NA)) {
                        int xs;
                        uint32_t xph;
                        ring_pos<NX>(i - NA, xs, xph);
                        if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&x_empty[xs], xph, abort_flag))) {
                            ok = false;
                            break;
                        }
                    }
                    ptx::tc_fence_after_sync();
                    ptx::tmem_st_32x32b_x32(tmem_base + lane_addr + kAStageCol + 64u * static_cast<uint32_t>(i % NA) + 32u * grp, a);
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&x_full[i % NX]);
                }
            }
        }
    } else if (kEpi && warp >= kWarpEpi0) {
        // ---------------------------------------------------------------- epilogue with bias, activation, gate, residual
        test_delay(kDelayEpilogue);   // the checked build can hold this role back (qlinear_test_delay)
        if constexpr (kEpi) {
            ptx::more_registers<kEpiRegs>();
            const int e = warp - kWarpEpi0;
            epilogue_role<kBf16Out, kAct>(p, ptx::smem_addr(smem + C::kOffEpi) + e * C::kNB * C::kStageBytes, C::kStageBytes,
                                          ptx::smem_addr(smem + C::kOffVec) + e * 2 * kEpiVectorBytes, tmem_base, acc_full,
                                          acc_empty, abort_flag, warp & 3, e >> 2, lane);
        }
    } else if (!give_registers<kEpi>()) {
    } else if (kLora && warp == kWarpTmaX) {
        // ---------------------------------------------------------------- activation producer, adapter mode
        test_delay(kDelayActivations);   // the checked build can hold this role back (qlinear_test_delay)
        // As the TMA producer below, by a whole warp.  An extra K-step's tile is 192 tokens x 64 columns: a row's own
        // parts of tw at its adapter's place in the tile's list, zero elsewhere.  Eight rows of one adapter (or none,
        // whose tw is zero) are a box of tw shifted by that place, and the TMA's fill past either end of tw's row gives
        // the zeros; 24 lanes issue a box each.  Eights with several adapters (where two requests meet, or tokens in
        // no order) are copied by the warp, in the layout the TMA writes: 128-byte rows, 16-byte pieces permuted by
        // the row's number mod 8.  All of a step's copies are on their way at once, and a step is announced when the
        // next one's are (290 rows of 38 requests one after the other, rank 64, a 128 -> 224 pair: 43 us, by loads and
        // stores 102; by the epilogue warps while they wait for the tile 32, but a layer with long prompts took 3 %
        // longer).  Tokens in no order make every eight such a one, 3 us a step: 290 rows of 38 adapters, rank 64,
        // 128 -> 224: 232 us; 4608 rows of 30 adapters, rank 16, 4608 -> 4608: 385 us, the same rows in order 205.
        if constexpr (kLora) {
            constexpr int kEights = BT / 8;
            uint32_t i = 0;
            bool ok = true;
            ptx::grid_dependency_wait();
            const int width = 2 * p.parts;                     // 16-byte pieces of a row of tw
            for (int un = blockIdx.x; un < num_units && ok; un += gridDim.x) {
                int t, kb0, kb1, p0, p1;
                unit(un, t, kb0, kb1);
                int t_blk, w_blk;
                tile_coords(t, p.num_w, t_blk, w_blk);
                lora_parts(un, t_blk, p0, p1);
                int own[BT / 32];                              // place of the adapter of row 32 j + lane, or -1
                int eight = -1;                                // lane l < 24: the place shared by rows 8 l .. 8 l + 7
                uint32_t mixed = 0;                            // the eights without one
#pragma unroll
                for (int j = 0; j < BT / 32; ++j) {
                    const int m = t_blk * BT + 32 * j + lane;
                    own[j] = p0 < p1 && m < p.M ? p.row_slot[m] : -1;
                    int top = own[j];
                    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    const uint32_t differ = __ballot_sync(0xFFFFFFFFu, own[j] >= 0 && own[j] != top);
                    const int of_lane = __shfl_sync(0xFFFFFFFFu, top, 8 * (lane & 3));
                    if ((lane >> 2) == j) eight = of_lane;
                    for (int o = 0; o < 4; ++o)
                        if ((differ >> (8 * o)) & 0xFFu) mixed |= 1u << (4 * j + o);
                }
                for (int kb = kb0; kb < kb1; ++kb, ++i) {
                    int s;
                    uint32_t ph;
                    ring_pos<NX>(i, s, ph);
                    if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&x_empty[s], ph ^ 1, abort_flag))) { ok = false; break; }
                    if (lane == 0) {
                        ptx::mbar_arrive_expect_tx(&x_full[s], kXBytes);
                        ptx::tma_load_2d(smem + C::kOffX + s * kXBytes, &map_x, &x_full[s], kb * BK, t_blk * BT);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                const uint4* tw = reinterpret_cast<const uint4*>(p.tw) + static_cast<int64_t>(t_blk) * BT * width;
                int copied = -1;                               // the stage whose copies are not announced yet
                const auto announce = [&] {
                    ptx::fence_proxy_async_smem();             // visible to the MMAs' reads of shared memory
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&x_full[copied]);
                };
                for (; p0 < p1; p0 += 4, ++i) {
                    int s;
                    uint32_t ph;
                    ring_pos<NX>(i, s, ph);
                    if (!__all_sync(0xFFFFFFFFu, ptx::mbar_wait(&x_empty[s], ph ^ 1, abort_flag))) { ok = false; break; }
                    uint8_t* stage = smem + C::kOffX + s * kXBytes;
                    if (lane == 0) ptx::mbar_expect_tx(&x_full[s], 1024u * static_cast<uint32_t>(kEights - __popc(mixed)));
                    __syncwarp();
                    if (lane < kEights && !((mixed >> lane) & 1u))
                        ptx::tma_load_2d(stage + 1024 * lane, &p.map_tw, &x_full[s], 16 * p0 - 8 * width * max(eight, 0),
                                         t_blk * BT + 8 * lane);
                    const int c = lane & 7;
#pragma unroll
                    for (int j = 0; j < BT / 32; ++j) {
                        for (uint32_t left = (mixed >> (4 * j)) & 15u; left != 0; left &= left - 1) {
                            const int e = __ffs(left) - 1;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {      // four rows at a time, eight lanes each
                                const int q = 8 * e + 4 * h + (lane >> 3);
                                const int slot = __shfl_sync(0xFFFFFFFFu, own[j], q);
                                const int rel = 2 * p0 + c - slot * width;
                                const bool in = slot >= 0 && static_cast<uint32_t>(rel) < static_cast<uint32_t>(width);
                                ptx::copy16_async(stage + (32 * j + q) * 128 + ((c ^ (q & 7)) << 4),
                                                  tw + (in ? (32 * j + q) * width + rel : 0), in);
                            }
                        }
                    }
                    if (mixed == 0) {
                        if (lane == 0) ptx::mbar_arrive(&x_full[s]);
                        continue;
                    }
                    ptx::copy_async_commit();
                    if (copied >= 0) {
                        ptx::copy_async_wait<1>();
                        announce();
                    }
                    copied = s;
                }
                if (copied >= 0) {
                    ptx::copy_async_wait<0>();
                    announce();
                }
            }
            if (lane == 0) {
                for (uint32_t j = (i > static_cast<uint32_t>(NX) ? i - NX : 0u); j < i; ++j)
                    ptx::mbar_wait(&x_full[j % NX], (j / NX) & 1u, nullptr);
            }
        }
    } else if (warp == kWarpTmaX) {
        // ---------------------------------------------------------------- TMA producer of activation tiles
        test_delay(kDelayActivations);   // the checked build can hold this role back (qlinear_test_delay)
        if (lane == 0) {
            uint32_t i = 0;
            bool ok = true;
            ptx::grid_dependency_wait();               // the activations come from the prepass
            for (int un = blockIdx.x; un < num_units && ok; un += gridDim.x) {
                int t, kb0, kb1;
                unit(un, t, kb0, kb1);
                int t_blk, w_blk;
                tile_coords(t, p.num_w, t_blk, w_blk);
                for (int kb = kb0; kb < kb1; ++kb, ++i) {
                    int s;
                    uint32_t ph;
                    ring_pos<NX>(i, s, ph);
                    if (!ptx::mbar_wait(&x_empty[s], ph ^ 1, abort_flag)) { ok = false; break; }
                    ptx::mbar_arrive_expect_tx(&x_full[s], kXBytes);
                    ptx::tma_load_2d(smem + C::kOffX + s * kXBytes, &map_x, &x_full[s], kb * BK, t_blk * BT);
                }
            }
            // Never leave the CTA with bulk copies still landing in its shared memory:
            // wait for the most recent load of every stage that received one.
            for (uint32_t j = (i > static_cast<uint32_t>(NX) ? i - NX : 0u); j < i; ++j)
                ptx::mbar_wait(&x_full[j % NX], (j / NX) & 1u, nullptr);
        }
    } else if (warp == kWarpTmaC) {
        // ---------------------------------------------------------------- TMA producer of codes and parameters
        test_delay(kDelayCodes);   // the checked build can hold this role back (qlinear_test_delay)
        // (the checked build's stall hook holds it back: no code or parameter load)
        if (lane == 0 && !stalled(kStallFused)) {
            // one code stage: kS K-steps of a tile's 256 rows (in SwiGLU mode 128 gate rows, then the same
            // 128 rows of the up weight); steps past the tensor's K are zero-filled, steps of the next
            // split-K slice are loaded and not used
            auto load_codes = [&](uint8_t* dst, uint64_t* bar, int kc, int w_blk) {
                if constexpr (kSwiGLU) {
                    ptx::tma_load_2d(dst, &map_codes, bar, kc * kCodeWords, w_blk * BWG);
                    ptx::tma_load_2d(dst + C::kCBytes / 2, &map_codes2, bar, kc * kCodeWords, w_blk * BWG);
                } else {
                    ptx::tma_load_2d(dst, &map_codes, bar, kc * kCodeWords, w_blk * BW);
                }
            };
            // The parameter pairs come from the prepass (the transpose, whose completion the conversion
            // just before this kernel on the stream implies; programmatic dependent launch): the code
            // loads of the first NC stages go out at once, their parameter loads (same stage barrier)
            // once the prepass is done.
            uint32_t ci = 0;
            bool ok = true, waited = false;
            int first_kc[NC], first_w[NC];
            auto late_params = [&] {
                ptx::grid_dependency_wait();
#pragma unroll
                for (int e = 0; e < NC; ++e)
                    if (static_cast<uint32_t>(e) < ci)
                        ptx::tma_load_2d(smem + C::kOffP + e * C::kPBytes, &map_params, &c_full[e], first_w[e] * BW,
                                         first_kc[e]);
                waited = true;
            };
            for (int un = blockIdx.x; un < num_units && ok; un += gridDim.x) {
                int t, kb0, kb1;
                unit(un, t, kb0, kb1);
                int t_blk, w_blk;
                tile_coords(t, p.num_w, t_blk, w_blk);
                for (int kc = kb0; kc < kb1; kc += C::kS, ++ci) {
                    int s;
                    uint32_t ph;
                    ring_pos<NC>(ci, s, ph);
                    if (ci >= static_cast<uint32_t>(NC) && !waited) late_params();
                    if (!ptx::mbar_wait(&c_empty[s], ph ^ 1, abort_flag)) { ok = false; break; }
                    ptx::mbar_arrive_expect_tx(&c_full[s], C::kCBytes + C::kPBytes);
                    load_codes(smem + C::kOffC + s * C::kCBytes, &c_full[s], kc, w_blk);
                    if (waited) {
                        ptx::tma_load_2d(smem + C::kOffP + s * C::kPBytes, &map_params, &c_full[s], w_blk * BW, kc);
                    } else {
#pragma unroll
                        for (int e = 0; e < NC; ++e) {     // constant indices keep the arrays in registers
                            if (e == s) {
                                first_kc[e] = kc;
                                first_w[e] = w_blk;
                            }
                        }
                    }
                }
                if constexpr (kLora) {
                    // a code stage per extra K-step: a box of B for each adapter (and projection) the step meets
                    if (!waited) late_params();
                    int p0, p1;
                    lora_parts(un, t_blk, p0, p1);
                    const int cols = part_cols(p.r8);
                    for (; ok && p0 < p1; p0 += 4, ++ci) {
                        int s;
                        uint32_t ph;
                        ring_pos<NC>(ci, s, ph);
                        const int seg0 = p0 / p.r8, seg1 = (min(p0 + 4, p1) - 1) / p.r8;
                        const uint32_t box_bytes = static_cast<uint32_t>((kSwiGLU ? BWG : BW) * cols * 2);
                        if (!ptx::mbar_wait(&c_empty[s], ph ^ 1, abort_flag)) { ok = false; break; }
                        ptx::mbar_arrive_expect_tx(&c_full[s], (seg1 - seg0 + 1) * box_bytes);
                        for (int seg = seg0; seg <= seg1; ++seg) {
                            const int up = kSwiGLU ? seg & 1 : 0;
                            const int adapter = p.tile_list[t_blk * BT + (kSwiGLU ? seg >> 1 : seg)];
                            uint8_t* dst = smem + C::kOffC + s * C::kCBytes + (seg - seg0) * (BW * cols * 2) + up * box_bytes;
                            ptx::tma_load_3d(dst, &p.map_b[up], &c_full[s], seg == seg0 ? 8 * (p0 - seg0 * p.r8) : 0,
                                             w_blk * (kSwiGLU ? BWG : BW), adapter);
                        }
                    }
                }
            }
            if (!waited) late_params();                // fewer than NC stages in all
            for (uint32_t j = (ci > static_cast<uint32_t>(NC) ? ci - NC : 0u); j < ci; ++j)
                ptx::mbar_wait(&c_full[j % NC], (j / NC) & 1u, nullptr);
        }
    } else if (warp == kWarpMma || warp == kWarpMma2) {
        // ---------------------------------------------------------------- MMA issuers, one per group
        test_delay(kDelayMma);   // the checked build can hold this role back (qlinear_test_delay)
        const int gsel = warp == kWarpMma ? 0 : 1;
        if (lane == 0) {
            constexpr uint32_t idesc = ptx::idesc_f16(BWG, BT, false);
            uint32_t i = 0;
            bool ok = true;
            int j = 0;
            for (int un = blockIdx.x; un < num_units && ok; un += gridDim.x, ++j) {
                int t, kb0, kb1;
                unit(un, t, kb0, kb1);
                for (int kb = kb0; kb < kb1; ++kb, ++i) {
                    int xs;
                    uint32_t xph;
                    ring_pos<NX>(i, xs, xph);
                    const int as = static_cast<int>(i % NA);
                    if (!ptx::mbar_wait(&x_full[xs], xph, abort_flag)) { ok = false; break; }   // x and A of step i
                    ptx::tc_fence_after_sync();
                    const uint32_t x_addr = ptx::smem_addr(smem + C::kOffX + xs * kXBytes);
                    {
                        const int g = gsel;
                        if (kb == kb0) {
                            // the previous unit's group-g results must have been drained
                            if (!ptx::mbar_wait(&acc_empty[g], (j & 1) ^ 1, abort_flag)) { ok = false; break; }
                            ptx::tc_fence_after_sync();
                        }
                        const uint32_t d = tmem_base + kAccCol + static_cast<uint32_t>(g * BT);
                        const uint32_t a_tm = tmem_base + kAStageCol + 64u * as + 32u * g;
#pragma unroll
                        for (int u = 0; u < BK / UK; ++u) {
                            ptx::mma_f16_ts(d, a_tm + u * (UK / 2), ptx::sdesc_sw128(x_addr + u * UK * 2), idesc,
                                            ((kb - kb0) | u) != 0);
                        }
                    }
                    if (!ok) break;
                    ptx::mma_commit(&x_empty[xs]);         // releases the x stage and the A stage
                }
                if constexpr (kLora) {
                    ptx::grid_dependency_wait();
                    constexpr uint32_t idesc_lora = ptx::idesc_f16(BWG, BT, true);
                    int t_blk, w_blk;
                    tile_coords(t, p.num_w, t_blk, w_blk);
                    int p0, p1;
                    lora_parts(un, t_blk, p0, p1);
                    for (; ok && p0 < p1; p0 += 4, ++i) {
                        int xs;
                        uint32_t xph;
                        ring_pos<NX>(i, xs, xph);
                        if (!ptx::mbar_wait(&x_full[xs], xph, abort_flag)) { ok = false; break; }
                        ptx::tc_fence_after_sync();
                        const uint32_t x_addr = ptx::smem_addr(smem + C::kOffX + xs * kXBytes);
                        const uint32_t d = tmem_base + kAccCol + static_cast<uint32_t>(gsel * BT);
                        const uint32_t a_tm = tmem_base + kAStageCol + 64u * static_cast<uint32_t>(i % NA) + 32u * gsel;
                        const int nu = min(BK / UK, p1 - p0);               // one 16-column MMA per part
                        int seg = p0 / p.r8, part = p0 - seg * p.r8;
                        for (int u = 0; u < nu; ++u) {
                            // the gate's and the up's parts each for their own row group: a zero operand under
                            // the other would turn an infinite t of one projection into a NaN of both
                            if (!kSwiGLU || (seg & 1) == gsel)
                                ptx::mma_f16_ts(d, a_tm + u * (UK / 2), ptx::sdesc_sw128(x_addr + u * UK * 2), idesc_lora, 1u);
                            if (kSwiGLU && ++part == p.r8) {
                                part = 0;
                                ++seg;
                            }
                        }
                        ptx::mma_commit(&x_empty[xs]);                      // (with no MMA of its own: of those before)
                    }
                }
                if (ok) ptx::mma_commit(&acc_full[0]);
            }
            // Wait until every MMA this thread issued has finished before TMEM is released.
            ptx::mma_commit(drain + gsel);
            ptx::mbar_wait(drain + gsel, 0, nullptr);
        }
    } else if (kSwiGLU && warp >= kWarpEpi0) {
        // ---------------------------------------------------------------- SwiGLU epilogue
        test_delay(kDelayEpilogue);   // the checked build can hold this role back (qlinear_test_delay)
        // Warp (quarter, half) reads the gate and up accumulators of TMEM lanes 32*quarter .. +31 (its
        // 32 intermediate columns) for the token chunks kHalfChunks*half .. +kHalfChunks-1.
        constexpr int kHalfChunks = BT / 32 / 2;
        const int quarter = warp & 3;
        const int half = (warp - kWarpEpi0) >> 2;
        uint8_t* epi_stage = smem + C::kOffEpi + (warp - kWarpEpi0) * C::kNB * C::kStageBytes;
        uint32_t nstore = 0;
        int j = 0;
        ptx::grid_dependency_wait();               // the row scales come from the kernels before this one
        for (int t = blockIdx.x; t < num_tiles; t += gridDim.x, ++j) {
            int t_blk, w_blk;
            tile_coords(t, p.num_w, t_blk, w_blk);
            // rs[c] belongs to token t_blk*BT + 32*(kHalfChunks*half + c) + lane
            float rs[kHalfChunks];
#pragma unroll
            for (int c = 0; c < kHalfChunks; ++c) {
                const int m = t_blk * BT + 32 * (kHalfChunks * half + c) + lane;
                rs[c] = (m < p.M) ? p.rowscale[m] : 0.0f;
            }
            const bool got = ptx::mbar_wait(&acc_full[0], j & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) break;
            ptx::tc_fence_after_sync();
            const int n_base = w_blk * BWG + quarter * 32;      // this warp's 32 intermediate columns
            const uint32_t tgate = tmem_base + kAccCol + (static_cast<uint32_t>(quarter * 32) << 16);
            const uint32_t tup = tgate + static_cast<uint32_t>(BT);
#pragma unroll
            for (int c = 0; c < kHalfChunks; ++c) {
                const int chunk = kHalfChunks * half + c;
                uint32_t rg[32], ru[32];
                ptx::tmem_ld_32x32b_x32(tgate + chunk * 32, rg);
                ptx::tmem_ld_32x32b_x32(tup + chunk * 32, ru);
                ptx::tmem_wait_ld();
                uint8_t* stage = epi_stage + (nstore % C::kNB) * C::kStageBytes;
                if (lane == 0) ptx::bulk_wait_group_read<C::kNB - 1>();   // the store that used this buffer has read it
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float sc = __shfl_sync(0xFFFFFFFFu, rs[c], k);
                    const float gv = __uint_as_float(rg[k]) * sc;
                    const float uv = __uint_as_float(ru[k]) * sc;
                    // the hardware exponential and reciprocal (a few fp32 ulps, far inside the bf16
                    // rounding that follows); -inf gives NaN and large negative g gives -0 as before
                    const float h = __fdividef(gv, 1.0f + __expf(-gv)) * uv;
                    if constexpr (kBf16Out) {
                        reinterpret_cast<__nv_bfloat16*>(stage)[k * 32 + lane] = __float2bfloat16_rn(h);
                    } else {
                        reinterpret_cast<float*>(stage)[k * 32 + lane] = h;
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::tma_store_2d(&map_y, stage, n_base, t_blk * BT + chunk * 32);
                    ptx::bulk_commit_group();
                }
                ++nstore;
            }
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&acc_empty[0]);
                ptx::mbar_arrive(&acc_empty[1]);
            }
        }
        if (lane == 0) ptx::bulk_wait_group_all();   // every store has completed before the CTA exits
    } else if (warp >= kWarpEpi0) {
        // ---------------------------------------------------------------- epilogue
        test_delay(kDelayEpilogue);   // the checked build can hold this role back (qlinear_test_delay)
        // All 8 warps drain group 0's accumulator first, then group 1's: warp (quarter, half) takes TMEM
        // lanes 32*quarter .. +31 and the token chunks kHalf*half .. +kHalf-1 of each group, so group 0 is
        // released after half a drain and its MMAs of the next unit run while group 1 is drained.
        constexpr int kHalf = BT / 32 / 2;         // token chunks of 32 per warp and group
        const int quarter = warp & 3;              // TMEM lanes 32*quarter .. +31
        const int half = (warp - kWarpEpi0) >> 2;
        uint8_t* epi_stage = smem + C::kOffEpi + (warp - kWarpEpi0) * C::kNB * C::kStageBytes;
        uint32_t nstore = 0;
        int j = 0;
        ptx::grid_dependency_wait();               // the row scales come from the kernels before this one
        for (int un = blockIdx.x; un < num_units; un += gridDim.x, ++j) {
            int t, kb0, kb1;
            unit(un, t, kb0, kb1);
            int t_blk, w_blk;
            tile_coords(t, p.num_w, t_blk, w_blk);
            // Row scales of this warp's tokens, fetched before the accumulators are ready:
            // rs[c] belongs to token t_blk*BT + 32*(kHalf*half + c) + lane.
            float rs[kHalf];
#pragma unroll
            for (int c = 0; c < kHalf; ++c) {
                const int m = t_blk * BT + 32 * (kHalf * half + c) + lane;
                rs[c] = (m < p.M) ? p.rowscale[m] : 0.0f;
            }
            const bool got = ptx::mbar_wait(&acc_full[0], j & 1, abort_flag);
            if (!__all_sync(0xFFFFFFFFu, got)) break;
            ptx::tc_fence_after_sync();
#pragma unroll 1
            for (int g = 0; g < NG; ++g) {
                const int n_base = w_blk * BW + g * BWG + quarter * 32;   // this warp's 32 output columns
                const uint32_t taddr = tmem_base + kAccCol + static_cast<uint32_t>(g * BT + 32 * kHalf * half) +
                                       (static_cast<uint32_t>(quarter * 32) << 16);
                // Two register buffers: the TMEM load of chunk c+1 is in flight while chunk c is stored.
                uint32_t r[2][32];
                ptx::tmem_ld_32x32b_x32(taddr, r[0]);
#pragma unroll
                for (int c = 0; c < kHalf; ++c) {
                    const int chunk = kHalf * half + c;
                    ptx::tmem_wait_ld();
                    if (c + 1 < kHalf) ptx::tmem_ld_32x32b_x32(taddr + (c + 1) * 32, r[(c + 1) & 1]);
                    const uint32_t* v = r[c & 1];
                    // staging block [32 tokens][32 columns], C::kNB of them per warp
                    uint8_t* stage = epi_stage + (nstore % C::kNB) * C::kStageBytes;
                    if (lane == 0) ptx::bulk_wait_group_read<C::kNB - 1>();   // the store that used this buffer has read it
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float val = __uint_as_float(v[k]) * __shfl_sync(0xFFFFFFFFu, rs[c], k);
                        if constexpr (kBf16Out) {
                            reinterpret_cast<__nv_bfloat16*>(stage)[k * 32 + lane] = __float2bfloat16_rn(val);
                        } else {
                            reinterpret_cast<float*>(stage)[k * 32 + lane] = val;
                        }
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kSplitK) {
                            ptx::tma_store_3d(&map_y, stage, n_base, t_blk * BT + chunk * 32, un / num_tiles);
                        } else {
                            ptx::tma_store_2d(&map_y, stage, n_base, t_blk * BT + chunk * 32);
                        }
                        ptx::bulk_commit_group();
                    }
                    ++nstore;
                }
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&acc_empty[g]);
            }
        }
        if (lane == 0) ptx::bulk_wait_group_all();   // every store has completed before the CTA exits
    }

    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace fused
}  // namespace ql
