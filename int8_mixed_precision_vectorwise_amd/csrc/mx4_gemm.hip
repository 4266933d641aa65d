// Product of two microscaled 4-bit matrices on gfx950's matrix cores:
//   out[i, j] = sum_k a[i, k] b[j, k] + bias[j],   a [m x k], b [n x k],
// with v_mfma_scale_f32_32x32x64_f8f6f4: E2M1 operands in blocks of 32 along k,
// each with its power of two, products exact and sums in fp32 (checked: within
// 2^-24 of the sum of magnitudes; a scale byte of 255 gives NaN).
//
// A lane of the instruction holds 32 codes (16 bytes) of one row and that block's
// scale; lane l has row l % 32 and block l / 32 of the step.  Which blocks of k meet
// in a step does not matter as long as both operands agree: of 128 elements, lanes
// 0..31 take blocks 0 and 1, lanes 32..63 blocks 2 and 3, in two steps.  A lane's two
// scales are then neighbouring bytes, the instruction picks the step's, and matrices
// lie in memory as plain rows.
//
// Workgroups of four waves, 2 x 2, each with 32 FM x 32 FN sums.  Stages of 256
// elements go from memory to LDS by direct loads, two places in turn: 128 bytes of
// codes a row are whole lines, which the L2 hands out at 134 GB/s a CU, lines halved
// (stages of 128 elements) at 70.  Scales come for two stages at once, 16 bytes a row: a
// load costs the vector memory path a cycle a row however few bytes it takes (with
// every stage of 128 elements, 4 bytes a row, they cost as much there as the codes).
// A stage is multiplied in quarters:
//   1  the second half's operands are read from LDS; then all waves have read the stage
//   2  its place fills with the stage after next; then all waves' share of the next is in
//   3, 4  the next stage's first half is read, the rest of the loads go out
// with reads and loads spread between the matrix instructions: a wave alone on its SIMD
// that waits for the load path to take another load starves the matrix cores (all loads
// in a row: 1.04 us for 128 elements of a 256 x 256 tile, spread 0.89, none 0.70).  The
// weights are the instruction's first operand: a lane then has four neighbouring columns
// of one output row.
//
// 256 x 256 tiles run 256 workgroups that take tiles in turn; a tile's first loads go
// out before the results of the one before it leave.  At 8192 x 8192 x 16384 the matrix
// cores are busy 59 % of the cycles at 1.76 GHz: the chip's power limit, which lets
// matrix instructions alone run at 1.79 GHz (6.4 PFLOP/s), leaves little to gain by more
// overlap.  The 16x16x128 instruction reaches 7.2 PFLOP/s alone, but its 64 accumulators
// of four registers left the compiler no room (100 registers spilled).
//
// Those tiles keep 103 to 134 scalar registers in lanes of vector registers (two tiles' descriptors and the products'
// arguments are alive at once); the smaller ones keep none.
//
// A tile's results pass through LDS: the bias of its columns waits in registers (read from
// LDS beside them it cost 2 us a tile), whole tiles leave by one address and fixed steps.
//
// Measured (fp16 out, operands of random numbers, us): 4096 x 22016 x 8192 376 in two
// launches (3.9 PFLOP/s), 8192 x 8192 x 16384 505 (4.4), 8192 x 8192 x 512 42, 512 x 4096 x
// 1024 5.7, bound by the launch and the latency of four stages.
#include <cmath>

#include "common.h"
#include "mx4.h"
#include "mx4_util.h"

namespace i8mp {

namespace {

constexpr int kStageK = 256;             // elements of a stage
constexpr int kRowBytes = kStageK / 2;   // its codes of a row: whole lines of the L2
constexpr int kXcds = 8, kCUs = 256;

// Whole tiles' results are stored through the L2: what is left in it is written back before a launch ends, which costs 1.6
// to 2.5 us, and the next launch finds them in the last-level cache either way.  us of a product, and with a scaling of
// its output after it, stored through / left in L2 / past the last-level cache:
//   2048 x 4096 x  512 (16 MiB)    7.9 / 9.5 / 8.8      18.3 / 20.1 / 19.0
//   4096 x 4096 x 2048 (32 MiB)    23.9 / 26.0 / 24.1   34.9 / 36.5 / 37.4
//   8192 x 8192 x  512 (128 MiB)   42.4 / 45.6 / 47.6   82.2 / 83.0 / 89.1
//   4096 x 22016 x 8192 (172 MiB)  366 / 367 / 360      443 / 438 / 451
//   5000 x 22016 x 1000 (210 MiB)  99 / 109 / 103       191 / 188 / 186
//   6607 x 22016 x 384 (277 MiB)   107 / 98 / 95        212 / 211 / 202
constexpr int kThrough = 16, kPast = 2;          // the stores' cache policies
constexpr int64_t kPastBytes = 256 << 20;        // the last-level cache: larger outputs pass it by

// lane i's 16 bytes at `offset` land at lds + 16 i (lds is the same in every lane)
__device__ inline void copy16(__amdgpu_buffer_rsrc_t src, uint8_t* lds, int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, offset, 0, 0, 0);
}

// accesses of LDS by the lanes of one wave stay on their side (LDS serves a wave in order)
__device__ inline void rows_done() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_wave_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Tile of a workgroup.  Workgroups go to the XCDs in turn; each XCD gets a run of
// neighbouring tiles, in groups of 8 tile rows, so that its L2 serves them.
__device__ inline void tile_of(uint32_t id, uint32_t count, uint32_t tiles_m, uint32_t tiles_n, int& tm, int& tn) {
    constexpr uint32_t kGroup = 8;
    const uint32_t full = count / kXcds * kXcds;
    const uint32_t t = id < full ? id % kXcds * (full / kXcds) + id / kXcds : id;
    const uint32_t group = t / (kGroup * tiles_n), first = group * kGroup, in = t - group * (kGroup * tiles_n);
    const uint32_t size = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    // divided by vector instructions: back to scalars, which the buffers' descriptors must be
    const uint32_t col = __builtin_amdgcn_readfirstlane(in / size);
    tm = __builtin_amdgcn_readfirstlane(first + (in - col * size));
    tn = col;
}

// until at most N of the wave's loads are under way, and its LDS reads are done
template <int N>
__device__ inline void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);
}

__device__ inline void meet() {
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
}

template <int FM, int FN>
struct Tile {
    static constexpr int BM = 64 * FM, BN = 64 * FN;
    static constexpr int kStage = (BM + BN) * kRowBytes;    // codes of a stage in LDS, a's first
    static constexpr int kScales = (BM + BN) * 16;          // scales of two stages
    static constexpr int kLoads = (BM + BN) / 32;           // a wave's loads of a stage's codes, 8 rows each
    static constexpr int kScaleLoads = (BM / 64 + 3) / 4;   // and of a's or b's scales, 64 rows each
    static_assert(BM >= BN, "b has no more rows than a");
    // The next tile's first stages are on their way while a tile's results leave, where one workgroup fills a CU
    static constexpr bool kAhead = FM * FN > 8;
    static constexpr int kRowOut = 128;                     // bytes of an output row that a wave stages at a time, at most
    static constexpr int kOutArea = 32 * (kRowOut + 16);    // 32 rows
    static constexpr int kScaleAt = 2 * kStage;
    static constexpr int kLds = kScaleAt + kScales + 2 * BN * 4 + (kAhead && 4 * kOutArea > kScales ? 4 * kOutArea : kScales);
};

// kPair: the workgroups from split on belong to a second product
template <int FM, int FN, int kType, bool kPair>
__global__ __launch_bounds__(256, FM * FN > 8 ? 1 : 2) void mx4_gemm_kernel(MxGemmArgs first, MxGemmArgs second, uint32_t split) {
    const bool later = kPair && blockIdx.x >= split;
    const MxGemmArgs& g = later ? second : first;
    const uint32_t block = later ? blockIdx.x - split : blockIdx.x, stride = !kPair ? gridDim.x : later ? gridDim.x - split : split;
    using T = Tile<FM, FN>;
    constexpr int BM = T::BM, BN = T::BN;
    constexpr int kBiasAt = T::kScaleAt + (T::kAhead ? T::kScales : 2 * T::kScales);
    constexpr int kScale2At = T::kAhead ? kBiasAt + 2 * BN * 4 : T::kScaleAt + T::kScales;
    constexpr int kOutAt = T::kAhead ? kScale2At : 0;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::kLds];
    static_assert(!T::kAhead || kScale2At + T::kScales <= T::kLds, "the second scales fit where results pass");
    float* const bias = reinterpret_cast<float*>(smem + kBiasAt);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, hi = lane >> 5;
    const int wm = (wave & 1) * 32 * FM, wn = (wave >> 1) * 32 * FN;
    const int lda = (int)g.a.ldc, ldb = (int)g.b.ldc, lsa = (int)g.a.lds, lsb = (int)g.b.lds, all_m = (int)g.a.rows, all_n = (int)g.b.rows;
    const int kp = (int)g.a.kp();
    const uint32_t tiles_m = (uint32_t)((g.a.rows + BM - 1) / BM), tiles_n = (uint32_t)((g.b.rows + BN - 1) / BN);
    const uint32_t tiles = tiles_m * tiles_n, units = tiles * (uint32_t)g.parts;
    if (kPair && block >= units) return;   // its product has fewer tiles than workgroups

    // A load of codes: 8 rows of 128 bytes, lane i the 16-byte chunk at place i % 8 of row i / 8.  Place p of row r
    // holds chunk p ^ (r / 2 % 8): the 16 lanes that LDS serves at once, which want one chunk of different rows, then
    // find it in 16 different bank groups.
    const int place = lane >> 3, chunk = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
    const int va = place * lda + chunk * 16, vb = place * ldb + chunk * 16;
    const int ya = lane * lsa, yb = lane * lsb;
    const int past = chunk >= 4 ? kOut : 0;   // of a last stage of 128 elements

    struct Unit {   // a tile, or a part of its sums
        __amdgpu_buffer_rsrc_t ca, cb, sa, sb;
        int m0, n0, rows_m, rows_n, part, stages;
        bool cut;   // the last stage has 128 elements
    };
    auto open = [&](uint32_t id) {   // 256 rows of at most I8MP_MAX_LD bytes: offsets and ranges fit 32 bits
        Unit u;
        u.part = __builtin_amdgcn_readfirstlane(id / tiles);
        tile_of(id - u.part * tiles, tiles, tiles_m, tiles_n, u.m0, u.n0);
        u.m0 *= BM;
        u.n0 *= BN;
        u.rows_m = all_m - u.m0 < BM ? all_m - u.m0 : BM;
        u.rows_n = all_n - u.n0 < BN ? all_n - u.n0 : BN;
        const int from = u.part * g.part_stages * kStageK, left = kp - from;
        u.stages = (left + kStageK - 1) / kStageK < g.part_stages ? (left + kStageK - 1) / kStageK : g.part_stages;
        u.cut = left < u.stages * kStageK;
        // k = 0: one stage, of zeros, from empty ranges
        u.stages = kp > 0 ? u.stages : 1;
        const int codes = from / 2, scales = from / kMxBlock;
        u.ca = range_of(g.a.codes + (int64_t)u.m0 * lda + codes, kp > 0 ? (u.rows_m - 1) * lda + kp / 2 - codes : 0);
        u.cb = range_of(g.b.codes + (int64_t)u.n0 * ldb + codes, kp > 0 ? (u.rows_n - 1) * ldb + kp / 2 - codes : 0);
        u.sa = range_of(g.a.scales + (int64_t)u.m0 * lsa + scales, kp > 0 ? (u.rows_m - 1) * lsa + kp / kMxBlock - scales : 0);
        u.sb = range_of(g.b.scales + (int64_t)u.n0 * lsb + scales, kp > 0 ? (u.rows_n - 1) * lsb + kp / kMxBlock - scales : 0);
        return u;
    };
    // Loads for stages past the last are out of range: every wait counts the same loads.
    auto copy = [&](const Unit& u, int i, int t) {   // load i of this wave for stage t
        uint8_t* const dst = smem + (t & 1) * T::kStage;
        const int at = (t < u.stages ? t * kRowBytes : kOut) + (u.cut && t == u.stages - 1 ? past : 0);
        if (i < BM / 32) {
            const int c = i * 4 + wave;
            copy16(u.ca, dst + c * 1024, va + at + c * 8 * lda);
        } else {
            const int c = (i - BM / 32) * 4 + wave;
            copy16(u.cb, dst + BM * kRowBytes + c * 1024, vb + at + c * 8 * ldb);
        }
    };
    auto scales_at = [&](int t) { return smem + (t >> 1 & 1 ? kScale2At : T::kScaleAt); };
    // Scales of stages t and t + 1 (t even), of a or of b: those of a go out one stage before they are read, those of b
    // two, so that every stage issues as many loads.  Bytes past a row's end are its neighbour's, or zeros.
    // Where rows are few some loads are made twice: the same bytes again.
    auto copy_scales = [&](const Unit& u, bool of_b, int t) {
        const int at = t < u.stages ? t * 8 : kOut;
#pragma unroll
        for (int i = 0; i < T::kScaleLoads; ++i) {
            const int c = (i * 4 + wave) % (BM / 64), d = (i * 4 + wave) % (BN / 64);
            copy16(of_b ? u.sb : u.sa, scales_at(t) + (of_b ? BM / 64 + d : c) * 1024,
                   (of_b ? yb + d * 64 * lsb : ya + c * 64 * lsa) + at);
        }
    };
    auto begin = [&](const Unit& u) {   // the loads of a tile's first two stages
        copy_scales(u, false, 0);
        copy_scales(u, true, 0);
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) copy(u, i, 0);
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) copy(u, i, 1);
    };

    v4i x[2][2][FM], w[2][2][FN];   // operands: half of the stage, step
    int sx[2][FM], sw[2][FN];
    const int row_x = wm + l32, row_w = BM + wn + l32, swz = l32 >> 1 & 7;
    auto read = [&](int p, int h, int t) {
        const uint8_t* const src = smem + (t & 1) * T::kStage + ((4 * p + 2 * hi + h) ^ swz) * 16;
#pragma unroll
        for (int i = 0; i < FM; ++i) x[p][h][i] = *reinterpret_cast<const v4i*>(src + (row_x + 32 * i) * kRowBytes);
#pragma unroll
        for (int j = 0; j < FN; ++j) w[p][h][j] = *reinterpret_cast<const v4i*>(src + (row_w + 32 * j) * kRowBytes);
    };
    // A second half that is not there has codes of zero; the first half's scales do for it.
    auto read_scales = [&](const Unit& u, int p, int t) {
        const uint8_t* const src = scales_at(t) + (t & 1) * 8 + (p == 1 && !(u.cut && t == u.stages - 1) ? 4 : 0) + 2 * hi;
#pragma unroll
        for (int i = 0; i < FM; ++i) sx[p][i] = *reinterpret_cast<const uint16_t*>(src + (row_x + 32 * i) * 16);
#pragma unroll
        for (int j = 0; j < FN; ++j) sw[p][j] = *reinterpret_cast<const uint16_t*>(src + (row_w + 32 * j) * 16);
    };
    v16f acc[FM][FN];
#define I8MP_MULTIPLY(p, h)                                                                                          \
    _Pragma("unroll") for (int i = 0; i < FM; ++i)                                                                   \
        _Pragma("unroll") for (int j = 0; j < FN; ++j)                                                               \
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(w[p][h][j]), operand(x[p][h][i]),    \
                                                                       acc[i][j], 4, 4, h, sw[p][j], h, sx[p][i])

    begin(open(block));
    uint32_t turn = 0;
    for (uint32_t id = block; id < units; id += stride, turn ^= 1) {
        const Unit u = open(id);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = v16f{};
        float* const tile_bias = bias + turn * BN;
        for (int j = threadIdx.x; j < BN; j += 256) tile_bias[j] = g.bias && j < u.rows_n ? widen(g.bias, (int64_t)u.n0 + j, g.out_dtype) : 0.0f;
        wait_loads<T::kLoads>();   // stage 0 has landed; no results pass where the second scales go any more
        meet();
        copy_scales(u, true, 2);
        read(0, 0, 0);
        read_scales(u, 0, 0);
        read(0, 1, 0);
        constexpr int kEarly = T::kLoads / 2;
        int t = 0;
        do {
            // first quarter: read the second half
            read(1, 0, t);
            read_scales(u, 1, t);
            read(1, 1, t);
            I8MP_MULTIPLY(0, 0);
#pragma unroll
            for (int i = 0; i < FM + FN; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): this wave has read stage t
            meet();
            // second quarter: its place is free for stage t + 2
            copy_scales(u, t & 1, t & 1 ? t + 3 : t + 2);
#pragma unroll
            for (int i = 0; i < kEarly; ++i) copy(u, i, t + 2);
            I8MP_MULTIPLY(0, 1);
#pragma unroll
            for (int i = 0; i < kEarly + T::kScaleLoads; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x8, FM * FN > 8 ? 2 : 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            wait_loads<kEarly + T::kScaleLoads>();   // stage t + 1 has landed
            meet();
            // second half: read the next stage's first
            read(0, 0, t + 1);
            read_scales(u, 0, t + 1);
            read(0, 1, t + 1);
#pragma unroll
            for (int i = kEarly; i < T::kLoads; ++i) copy(u, i, t + 2);
            I8MP_MULTIPLY(1, 0);
            I8MP_MULTIPLY(1, 1);
#pragma unroll
            for (int i = 0; i < 3 * (FM + FN) / 2; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
#pragma unroll
            for (int i = 0; i < T::kLoads - kEarly; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, FM * FN > 8 ? 2 : 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        } while (++t < u.stages);
        wait_loads<0>();   // none lands in what follows
        meet();            // the stages are free
        if (T::kAhead && id + stride < units) begin(open(id + stride));

        // Sums (i, j, r): row wm + 32 i + l32, column wn + 32 j + 8 (r / 4) + 4 hi + r % 4.  They pass through the wave's
        // part of LDS, 32 rows of kCols at a time, and leave as 16-byte pieces of whole lines.
        constexpr int kElem = kType == I8MP_DTYPE_F32 ? 4 : 2;
        constexpr int kTiles = T::kRowOut / kElem / 32 < FN ? T::kRowOut / kElem / 32 : FN, kCols = 32 * kTiles;
        constexpr int kPitch = kCols * kElem + 16, kPieces = kCols * kElem / 16, kEach = 16 / kElem;
        uint8_t* const out = static_cast<uint8_t*>(g.out) + u.part * g.part_bytes;
        uint8_t* const area = smem + kOutAt + wave * T::kOutArea;
        const bool whole = g.ldout * kElem % 16 == 0 && reinterpret_cast<uintptr_t>(g.out) % 16 == 0;
        const bool all = whole && u.rows_m == BM && u.rows_n == BN;
        const int64_t pitch = g.ldout * kElem;
        const int row0 = wm + lane / kPieces, col0 = wn + lane % kPieces * kEach;   // of the lane's first piece
        const int at0 = row0 * (int)pitch + col0 * kElem;
        const __amdgpu_buffer_rsrc_t tile_to = range_of(out + u.m0 * pitch + u.n0 * (int64_t)kElem, (BM - 1) * (int)pitch + BN * kElem);
        uint8_t* const first_to = out + (u.m0 + row0) * pitch + (u.n0 + col0) * (int64_t)kElem;
        const uint8_t* const from = area + lane / kPieces * kPitch + lane % kPieces * 16;
#pragma unroll
        for (int j0 = 0; j0 < FN; j0 += kTiles) {
            v4f b[kTiles][4];
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) b[j][q] = *reinterpret_cast<const v4f*>(tile_bias + wn + 32 * (j0 + j) + 8 * q + 4 * hi);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                // so many sums at a time leave the accumulation registers
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (T::kAhead) {
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) asm volatile("" : "+a"(acc[i][j0 + j]));
                }
#pragma unroll
                for (int j = 0; j < kTiles; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int col = 32 * j + 8 * q + 4 * hi;
                        float v[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = acc[i][j0 + j][4 * q + r] + b[j][q][r];
                        uint8_t* p = area + l32 * kPitch + col * kElem;
                        if constexpr (kType == I8MP_DTYPE_F32) *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
                        else *reinterpret_cast<uint2*>(p) = make_uint2(narrow2<kType>(v[0], v[1]), narrow2<kType>(v[2], v[3]));
                    }
                rows_done();
#pragma unroll
                for (int v = 0; v < kPieces / 2; ++v) {
                    constexpr int kRows = 64 / kPieces;   // of 64 lanes
                    const v4u* const piece = reinterpret_cast<const v4u*>(from + v * kRows * kPitch);
                    uint8_t* const to = first_to + (32 * i + v * kRows) * pitch + 32 * j0 * kElem;
                    if (all) {
                        const int step = (32 * i + v * kRows) * (int)pitch + 32 * j0 * kElem;
                        if (g.past) __builtin_amdgcn_raw_buffer_store_b128(*piece, tile_to, at0, step, kPast);
                        else __builtin_amdgcn_raw_buffer_store_b128(*piece, tile_to, at0, step, kThrough);
                        continue;
                    }
                    const int r = row0 + 32 * i + v * kRows, c = col0 + 32 * j0;
                    if (r >= u.rows_m || c >= u.rows_n) continue;
                    if (whole && c + kEach <= u.rows_n) {
                        *reinterpret_cast<v4u*>(to) = *piece;
                    } else {
#pragma unroll
                        for (int e = 0; e < kEach; ++e) {
                            if (c + e >= u.rows_n) break;
                            if constexpr (kElem == 4) reinterpret_cast<uint32_t*>(to)[e] = reinterpret_cast<const uint32_t*>(piece)[e];
                            else reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(piece)[e];
                        }
                    }
                }
                rows_done();
            }
        }
        if constexpr (!T::kAhead) break;   // as many workgroups as units
    }
#undef I8MP_MULTIPLY
}

// out = sum over parts + bias, parts in order; four columns a lane
template <int kType>
__global__ __launch_bounds__(256) void mx4_join_kernel(MxGemmArgs g, const float* part, int64_t ldp) {
    const int64_t quads = ldp / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t r = i / quads, c = (i - r * quads) * 4;
    if (r >= g.a.rows) return;
    const float* p = part + r * ldp + c;
    v4f v = *reinterpret_cast<const v4f*>(p);
    for (int q = 1; q < g.parts; ++q) v += *reinterpret_cast<const v4f*>(p + q * g.part_bytes / 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (c + e >= g.b.rows) break;
        const float x = g.bias ? v[e] + widen(g.bias, c + e, kType) : v[e];
        const int64_t at = r * g.ldout + c + e;
        if constexpr (kType == I8MP_DTYPE_F32) static_cast<float*>(g.out)[at] = x;
        else static_cast<half_bits*>(g.out)[at] = (half_bits)narrow2<kType>(x, 0.0f);
    }
}

template <int F, int kType>
hipError_t launch_tiles(const MxGemmArgs& g, hipStream_t stream) {
    using T = Tile<F, F>;
    const int64_t units = ceil_div(g.a.rows, T::BM) * ceil_div(g.b.rows, T::BN) * g.parts;
    const dim3 grid((unsigned)(T::kAhead && units > kCUs ? kCUs : units));
    hipLaunchKernelGGL((mx4_gemm_kernel<F, F, kType, false>), grid, dim3(256), 0, stream, g, g, 0u);
    return hipGetLastError();
}
template <int F>
hipError_t launch_type(const MxGemmArgs& g, hipStream_t stream) {
    return g.out_dtype == I8MP_DTYPE_F32   ? launch_tiles<F, I8MP_DTYPE_F32>(g, stream)
           : g.out_dtype == I8MP_DTYPE_F16 ? launch_tiles<F, I8MP_DTYPE_F16>(g, stream)
                                           : launch_tiles<F, I8MP_DTYPE_BF16>(g, stream);
}
hipError_t launch_one(int f, const MxGemmArgs& g, hipStream_t stream) {
    return f == 4 ? launch_type<4>(g, stream) : f == 2 ? launch_type<2>(g, stream) : launch_type<1>(g, stream);
}

// ---- which tiles -----------------------------------------------------------------
// A cost model in us, fitted to timed products: a launch starts in 2; a tile of 64 f costs a
// fixed time, and a time a stage that depends on how many of them share a CU.
//   f   rows    a CU holds   fixed   a stage, with 1 .. of them on a CU
//   4   256     1            7       1.75
//   2   128     2            3       0.65  1.35
//   1   64      4            1.8     0.44  0.62  0.9  1.2
// Between one and two of 128 rows a CU the waiting ones help early: 1.08 with 352 on 256 CUs, 1.11 with 384.
// us with each shape alone, unsplit:  256 rows   128 rows   64 rows
//    512 x  8192 x  8192                  50.7       26.1      39.4
//    646 x  4096 x  5120                  33.9       15.7      20.1
//     64 x 13824 x  5120                  32.9       16.3      12.7
//   3663 x 22016 x  1435                   110        108       160
//   4096 x  4096 x  2048                  22.9       26.9      42.1
//   5673 x  5120 x 11008                   164        217       351
// Tiles of 256 x 128, one a CU, gain 8 to 14 % where they come to just one a CU, and nothing elsewhere: not kept.
constexpr int kShapes[3] = {4, 2, 1};
constexpr double kStart = 2.0;
double stage_us(int f, double on_cu) {
    static const double t1[] = {0.44, 0.62, 0.9, 1.2};
    return f == 4 ? 1.75 : f == 2 ? 0.65 + (on_cu > 1.0 ? 0.7 * std::sqrt(on_cu - 1.0) : 0.0) : t1[(int)std::ceil(on_cu) - 1];
}
double fixed_us(int f) { return f == 4 ? 7.0 : f == 2 ? 3.0 : 1.8; }
double tiles_us(int f, int64_t units, double stages) {
    const int64_t hold = f == 4 ? 1 : f == 2 ? 2 : 4;
    const int64_t full = units / (kCUs * hold), rest = units - full * kCUs * hold;
    return kStart + full * (fixed_us(f) + stages * stage_us(f, hold)) +
           (rest ? fixed_us(f) + stages * stage_us(f, (double)rest / kCUs) : 0.0);
}

struct Cut {   // of a product's columns: one tile shape, sums in `parts` parts of `part_stages`
    int f, parts;
    int64_t part_stages;
    double us;
};
// Sums are split over k where tiles alone leave CUs idle: the parts, in fp32, pass through the workspace, and a second
// launch adds them.
Cut best_cut(int64_t m, int64_t n, int64_t k) {
    const int64_t stages = ceil_div(k, kStageK) > 0 ? ceil_div(k, kStageK) : 1;
    Cut best{1, 1, stages, 1e300};
    for (int f : kShapes) {
        const int64_t tiles = ceil_div(m, 64 * f) * ceil_div(n, 64 * f);
        for (int parts = 1; parts <= 16 && parts <= stages; ++parts) {
            const int64_t per = ceil_div(stages, parts);
            if (ceil_div(stages, per) != parts) continue;
            if (parts > 1 && tiles * parts > 4 * kCUs) break;
            double us = tiles_us(f, tiles * parts, (double)per);
            // a second launch, on the host too, and the parts through the last-level cache at 10 TB/s
            if (parts > 1) us += 5.0 + 0.2 * parts + (double)m * n * 8 * parts / 1.0e7;
            if (us < best.us) best = Cut{f, parts, per, us};
        }
    }
    return best;
}
// A product too large for one round may take whole rounds of 256 x 256 tiles for its first columns and another cut for
// the rest, in a second launch.
struct Plan {
    int64_t n_main;   // 0: all columns by `rest`
    Cut rest;
    double us;
};
Plan plan(int64_t m, int64_t n, int64_t k) {
    const Cut whole = best_cut(m, n, k);
    Plan p{0, whole, whole.us};
    const int64_t rows = ceil_div(m, 256), rounds = rows * ceil_div(n, 256) / kCUs, cols = rounds * kCUs / rows;
    const int64_t n_main = cols * 256, stages = ceil_div(k, kStageK);
    if (cols > 0 && n_main < n) {
        const Cut rest = best_cut(m, n - n_main, k);
        const double us = tiles_us(4, rows * cols, (double)stages) + 1.0 + rest.us;
        if (us < 0.98 * whole.us) p = Plan{n_main, rest, us};
    }
    return p;
}
int64_t part_row(int64_t n) { return round_up(n, 4); }

}  // namespace

size_t mx4_gemm_workspace(int64_t m, int64_t n, int64_t k) {
    if (m <= 0 || n <= 0 || mx4_decode_fits(m, k)) return 0;
    const Plan p = plan(m, n, k);
    return p.rest.parts > 1 ? (size_t)p.rest.parts * m * part_row(n - p.n_main) * 4 : 0;
}

// Two products of one type in one launch, where the model finds that to beat one after the other:
// - by 64 x 64 tiles, all of them, those of the longer sums first.  Gradients of 512 x 4096 x 1024: 12.4 us, one
//   after the other 16.8.
// - by 256 x 256 tiles, a share of the workgroups each.  Gradients of 2048 x 4096 x 4096 (128 tiles of 16 stages, 256
//   of 8): 46.9 us, one after the other 52.3.
template <int F, int kType>
hipError_t launch_pair(const MxGemmArgs& x, const MxGemmArgs& y, int64_t split, int64_t all, hipStream_t stream) {
    hipLaunchKernelGGL((mx4_gemm_kernel<F, F, kType, true>), dim3((unsigned)all), dim3(256), 0, stream, x, y, (uint32_t)split);
    return hipGetLastError();
}

hipError_t launch_mx4_gemm_pair(const MxGemmArgs& a, const MxGemmArgs& b, hipStream_t stream) {
    MxGemmArgs x = a.a.k >= b.a.k ? a : b, y = a.a.k >= b.a.k ? b : a;
    for (MxGemmArgs* g : {&x, &y}) {
        g->parts = 1;
        g->part_stages = (int)ceil_div(g->a.k, kStageK);
        g->part_bytes = 0;
        g->past = g->a.rows * g->b.rows * 2 > kPastBytes;
    }
    const auto tiles = [](const MxGemmArgs& g, int f) { return ceil_div(g.a.rows, 64 * f) * ceil_div(g.b.rows, 64 * f); };
    const bool bf16 = x.out_dtype == I8MP_DTYPE_BF16;
    if (!mx4_decode_fits(x.a.rows, x.a.k) && !mx4_decode_fits(y.a.rows, y.a.k)) {
        const Plan px = plan(x.a.rows, x.b.rows, x.a.k), py = plan(y.a.rows, y.b.rows, y.a.k);
        double best = 0.98 * (px.us + 1.0 + py.us);
        const int64_t sx = tiles(x, 1), all = sx + tiles(y, 1);
        const double mean = ((double)sx * x.part_stages + (double)(all - sx) * y.part_stages) / all;
        const double longest = kStart + fixed_us(1) + x.part_stages * stage_us(1, 2.0), together = tiles_us(1, all, mean);
        const bool small = (longest > together ? longest : together) < best;
        if (small) best = longest > together ? longest : together;
        // whole XCDs' turns each: a workgroup's tiles stay on its XCD
        const int64_t tx = tiles(x, 4), ty = tiles(y, 4);
        int64_t split = 0;
        for (int64_t s = kXcds; s < kCUs; s += kXcds) {
            const double ux = tiles_us(4, ceil_div(tx, s) * kCUs, x.part_stages), uy = tiles_us(4, ceil_div(ty, kCUs - s) * kCUs, y.part_stages);
            if ((ux > uy ? ux : uy) < best) best = ux > uy ? ux : uy, split = s;
        }
        if (split > 0) return bf16 ? launch_pair<4, I8MP_DTYPE_BF16>(x, y, split, kCUs, stream) : launch_pair<4, I8MP_DTYPE_F16>(x, y, split, kCUs, stream);
        if (small) return bf16 ? launch_pair<1, I8MP_DTYPE_BF16>(x, y, sx, all, stream) : launch_pair<1, I8MP_DTYPE_F16>(x, y, sx, all, stream);
    }
    if (hipError_t e = launch_mx4_gemm(a, stream); e != hipSuccess) return e;
    return launch_mx4_gemm(b, stream);
}

hipError_t launch_mx4_gemm(const MxGemmArgs& args, hipStream_t stream) {
    if (mx4_decode_fits(args.a.rows, args.a.k)) return launch_mx4_decode(args, stream);
    const int64_t m = args.a.rows, n = args.b.rows, k = args.a.k, elem = args.out_dtype == I8MP_DTYPE_F32 ? 4 : 2;
    const Plan p = plan(m, n, k);
    MxGemmArgs g = args;
    g.parts = 1;
    g.part_stages = (int)ceil_div(k, kStageK);
    g.part_bytes = 0;
    g.past = m * n * elem > kPastBytes;
    if (p.n_main > 0) {
        g.b.rows = p.n_main;
        if (hipError_t e = launch_one(4, g, stream); e != hipSuccess) return e;
        g.b.rows = n - p.n_main;
        g.b.codes += p.n_main * g.b.ldc;
        g.b.scales += p.n_main * g.b.lds;
        g.out = static_cast<uint8_t*>(g.out) + p.n_main * elem;
        if (g.bias) g.bias = static_cast<const uint8_t*>(g.bias) + p.n_main * elem;
    }
    if (p.rest.parts == 1) return launch_one(p.rest.f, g, stream);
    const int64_t ldp = part_row(g.b.rows);
    MxGemmArgs s = g;   // the parts
    s.out = g.part;
    s.out_dtype = I8MP_DTYPE_F32;
    s.ldout = ldp;
    s.bias = nullptr;
    s.parts = g.parts = p.rest.parts;
    s.part_stages = (int)p.rest.part_stages;
    s.part_bytes = g.part_bytes = m * ldp * 4;
    s.past = false;
    if (hipError_t e = launch_one(p.rest.f, s, stream); e != hipSuccess) return e;
    const dim3 grid((unsigned)ceil_div(m * ldp / 4, 256));
    if (g.out_dtype == I8MP_DTYPE_F32) hipLaunchKernelGGL((mx4_join_kernel<I8MP_DTYPE_F32>), grid, dim3(256), 0, stream, g, g.part, ldp);
    else if (g.out_dtype == I8MP_DTYPE_F16) hipLaunchKernelGGL((mx4_join_kernel<I8MP_DTYPE_F16>), grid, dim3(256), 0, stream, g, g.part, ldp);
    else hipLaunchKernelGGL((mx4_join_kernel<I8MP_DTYPE_BF16>), grid, dim3(256), 0, stream, g, g.part, ldp);
    return hipGetLastError();
}

}  // namespace i8mp
