// Product of two microscaled 4-bit matrices on gfx950's matrix cores:
//   out[i, j] = sum_k a[i, k] b[j, k] + bias[j],   a [m x k], b [n x k],
// with v_mfma_scale_f32_32x32x64_f8f6f4: E2M1 operands in blocks of 32 along k,
// each with its power of two, products exact and sums in fp32 (checked: within
// 2^-24 of the sum of magnitudes; a scale byte of 255 gives NaN).
//
// A lane of the instruction holds 32 codes (16 bytes) of one row and that block's
// scale; lane l has row l % 32 and block l / 32 of the step.  Which blocks of k
// meet in a step does not matter as long as both operands agree, so a stage of 256
// elements is taken as four steps in which lanes 0..31 have blocks 0, 1, 2, 3 and
// lanes 32..63 blocks 4, 5, 6, 7: a lane's four scales are then one aligned word
// of the row, the instruction picks the step's byte, and the matrices need no
// other order in memory than rows.
//
// Workgroups of four waves, 2 x 2, each with 32 FM x 32 FN sums.  Stages of 256
// elements (128 bytes of codes and 8 of scales a row) go from memory to LDS by
// direct loads, two buffers in turn.  The weights are the instruction's first
// operand: a lane then has four neighbouring columns of one output row.
#include "common.h"
#include "mx4.h"

namespace i8mp {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kStageK = 256;             // elements of a stage
constexpr int kRowBytes = kStageK / 2;   // its codes of a row
constexpr int kXcds = 8;
constexpr int kOut = (int)0x80000000;    // a buffer offset past every range: reads zeros

__device__ inline __amdgpu_buffer_rsrc_t range_of(const void* base, int64_t bytes) {
    bytes = bytes < 0 ? 0 : bytes > 0x7fffffffLL ? 0x7fffffffLL : bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

// lane i's 16 or 4 bytes at `offset` land at lds + 16 i or 4 i (lds is the same in every lane)
__device__ inline void copy16(__amdgpu_buffer_rsrc_t src, uint8_t* lds, int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, offset, 0, 0, 0);
}
__device__ inline void copy4(__amdgpu_buffer_rsrc_t src, uint8_t* lds, int offset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 4, offset, 0, 0, 0);
}

__device__ inline v8i operand(const v4i& x) { return __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1); }

__device__ inline float widen(const void* p, int64_t i, int dtype) {
    if (dtype == I8MP_DTYPE_F32) return static_cast<const float*>(p)[i];
    const half_bits h = static_cast<const half_bits*>(p)[i];
    return dtype == I8MP_DTYPE_BF16 ? __uint_as_float((uint32_t)h << 16) : h2f(h);
}
template <int kType>
__device__ inline uint32_t narrow2(float x, float y) {
    if constexpr (kType == I8MP_DTYPE_BF16)
        return __builtin_bit_cast(half_bits, (__bf16)x) | (uint32_t)__builtin_bit_cast(half_bits, (__bf16)y) << 16;
    else return f2h(x) | (uint32_t)f2h(y) << 16;
}

// accesses of LDS by the lanes of one wave stay on their side (LDS serves a wave in order)
__device__ inline void rows_done() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_wave_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Tile of a workgroup.  Workgroups go to the XCDs in turn; each XCD gets a run of
// neighbouring tiles, in groups of 8 tile rows, so that its L2 serves them.
__device__ inline void tile_of(int64_t id, int64_t count, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn) {
    constexpr int kGroup = 8;
    const int64_t full = count / kXcds * kXcds;
    const int64_t t = id < full ? id % kXcds * (full / kXcds) + id / kXcds : id;
    const int64_t first = t / (kGroup * tiles_n) * kGroup, in = t % (kGroup * tiles_n);
    const int64_t size = tiles_m - first < kGroup ? tiles_m - first : kGroup;
    tm = first + in % size;
    tn = in / size;
}

template <int FM, int FN>
struct Tile {
    static constexpr int BM = 64 * FM, BN = 64 * FN;
    static constexpr int kCodes = (BM + BN) * kRowBytes;   // a stage in LDS: codes of a, of b, then the scales
    static constexpr int kStage = kCodes + (BM + BN) * 8;
    static constexpr int kCopies = (BM + BN) / 32;         // copies of codes a wave and stage, 8 rows each
    static constexpr int kScaleCopies = (BM + BN) / 128;   // of scales, 32 rows each
    static_assert((BM + BN) % 128 == 0, "the waves' shares of the copies are equal");
};

template <int FM, int FN, int kType>
__global__ __launch_bounds__(256, FM * FN > 8 ? 1 : 2) void mx4_gemm_kernel(MxGemmArgs g) {
    using T = Tile<FM, FN>;
    constexpr int BM = T::BM, BN = T::BN;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * T::kStage + BN * 4];
    float* const bias = reinterpret_cast<float*>(smem + 2 * T::kStage);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l32 = lane & 31, hi = lane >> 5;
    const int wm = (wave & 1) * 32 * FM, wn = (wave >> 1) * 32 * FN;
    int64_t tm, tn;
    tile_of(blockIdx.x, gridDim.x, (g.a.rows + BM - 1) / BM, (g.b.rows + BN - 1) / BN, tm, tn);
    const int64_t m0 = tm * BM, n0 = tn * BN, kp = g.a.kp();
    const int64_t rows_m = g.a.rows - m0 < BM ? g.a.rows - m0 : BM, rows_n = g.b.rows - n0 < BN ? g.b.rows - n0 : BN;
    const __amdgpu_buffer_rsrc_t ca = range_of(g.a.codes + m0 * g.a.ldc, (rows_m - 1) * g.a.ldc + kp / 2);
    const __amdgpu_buffer_rsrc_t cb = range_of(g.b.codes + n0 * g.b.ldc, (rows_n - 1) * g.b.ldc + kp / 2);
    const __amdgpu_buffer_rsrc_t sa = range_of(g.a.scales + m0 * g.a.lds, (rows_m - 1) * g.a.lds + kp / kMxBlock);
    const __amdgpu_buffer_rsrc_t sb = range_of(g.b.scales + n0 * g.b.lds, (rows_n - 1) * g.b.lds + kp / kMxBlock);
    const int stages = (int)((kp + kStageK - 1) / kStageK);
    const bool half = kp % kStageK != 0;   // the last stage has 128 elements

    // Copies of codes: 8 rows of 128 bytes each, lane i the 16-byte chunk at place i % 8 of row i / 8.
    // Place p of row r holds chunk p ^ (r / 2 % 8): the 16 lanes that LDS serves at once read one chunk of
    // 16 neighbouring rows, which then lie in 16 different bank groups.
    int place[2], chunk[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {   // copies of even and of odd index
        chunk[q] = (lane & 7) ^ ((4 * q + (lane >> 4)) & 7);
        place[q] = lane >> 3;
    }
    auto copy_codes = [&](int c, uint8_t* dst, int t, bool last) {   // copy c of a stage, a's first
        const int ld = (int)(c < BM / 8 ? g.a.ldc : g.b.ldc), row = (c < BM / 8 ? c : c - BM / 8) * 8;
        int off = (row + place[c & 1]) * ld + chunk[c & 1] * 16 + t * kRowBytes;
        if (last && half && chunk[c & 1] >= 4) off = kOut;
        copy16(c < BM / 8 ? ca : cb, dst + c * 1024, off);
    };
    auto copy_scales = [&](int c, uint8_t* dst, int t, bool last) {  // 32 rows of two words
        const int ld = (int)(c < BM / 32 ? g.a.lds : g.b.lds), row = (c < BM / 32 ? c : c - BM / 32) * 32;
        int off = (row + (lane >> 1)) * ld + (lane & 1) * 4 + t * 8;
        if (last && half && (lane & 1)) off = kOut;
        copy4(c < BM / 32 ? sa : sb, dst + T::kCodes + c * 256, off);
    };
    auto fill = [&](int t) {
        uint8_t* dst = smem + (t & 1) * T::kStage;
        const bool last = t == stages - 1;
#pragma unroll
        for (int i = 0; i < T::kCopies; ++i) copy_codes(i * 4 + wave, dst, t, last);
#pragma unroll
        for (int i = 0; i < T::kScaleCopies; ++i) copy_scales(i * 4 + wave, dst, t, last);
    };

    v16f acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    for (int j = threadIdx.x; j < BN; j += 256) bias[j] = g.bias && j < rows_n ? widen(g.bias, n0 + j, g.out_dtype) : 0.0f;

    if (stages > 0) fill(0);
    for (int t = 0; t < stages; ++t) {
        __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0): this wave's copies of stage t
        __syncthreads();
        if (t + 1 < stages) fill(t + 1);
        const uint8_t* src = smem + (t & 1) * T::kStage;
        int sx[FM], sw[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) sx[i] = *reinterpret_cast<const int*>(src + T::kCodes + ((wm + 32 * i + l32) * 2 + hi) * 4);
#pragma unroll
        for (int j = 0; j < FN; ++j) sw[j] = *reinterpret_cast<const int*>(src + T::kCodes + ((BM + wn + 32 * j + l32) * 2 + hi) * 4);
#define I8MP_STEP(s)                                                                                                  \
    do {                                                                                                              \
        v4i x[FM], w[FN];                                                                                             \
        const int at = ((4 * hi + s) ^ ((l32 >> 1) & 7)) * 16;                                                        \
        _Pragma("unroll") for (int i = 0; i < FM; ++i)                                                                \
            x[i] = *reinterpret_cast<const v4i*>(src + (wm + 32 * i + l32) * kRowBytes + at);                         \
        _Pragma("unroll") for (int j = 0; j < FN; ++j)                                                                \
            w[j] = *reinterpret_cast<const v4i*>(src + (BM + wn + 32 * j + l32) * kRowBytes + at);                    \
        _Pragma("unroll") for (int i = 0; i < FM; ++i)                                                                \
            _Pragma("unroll") for (int j = 0; j < FN; ++j)                                                            \
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(w[j]), operand(x[i]), acc[i][j], \
                                                                           4, 4, s, sw[j], s, sx[i]);                 \
    } while (0)
        I8MP_STEP(0);
        I8MP_STEP(1);
        I8MP_STEP(2);
        I8MP_STEP(3);
#undef I8MP_STEP
    }
    __syncthreads();   // the stages are free, the bias is there

    // Sums (i, j, r): row wm + 32 i + l32, column wn + 32 j + 8 (r / 4) + 4 hi + r % 4.  They pass through the
    // wave's part of LDS, 32 rows at a time, and leave as 16-byte pieces of whole rows.
    constexpr int kElem = kType == I8MP_DTYPE_F32 ? 4 : 2, kPitch = 32 * FN * kElem + 16;
    static_assert(4 * 32 * kPitch <= 2 * T::kStage, "the waves' rows fit the stages");
    uint8_t* const area = smem + wave * 32 * kPitch;
    const bool whole = g.ldout * kElem % 16 == 0 && reinterpret_cast<uintptr_t>(g.out) % 16 == 0;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = 32 * j + 8 * q + 4 * hi;
                const v4f b = *reinterpret_cast<const v4f*>(bias + wn + col);
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = acc[i][j][4 * q + r] + b[r];
                uint8_t* p = area + l32 * kPitch + col * kElem;
                if constexpr (kType == I8MP_DTYPE_F32) *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
                else *reinterpret_cast<uint2*>(p) = make_uint2(narrow2<kType>(v[0], v[1]), narrow2<kType>(v[2], v[3]));
            }
        rows_done();
        constexpr int kPieces = 32 * FN * kElem / 16, kEach = 16 / kElem;
#pragma unroll
        for (int u = 0; u < kPieces / 2; ++u) {
            const int p = u * 64 + lane, row = p / kPieces, col = p % kPieces * kEach;
            const int64_t r = wm + 32 * i + row, c = wn + col;
            if (r >= rows_m || c >= rows_n) continue;
            const uint8_t* from = area + row * kPitch + col * kElem;
            uint8_t* to = static_cast<uint8_t*>(g.out) + ((m0 + r) * g.ldout + n0 + c) * kElem;
            if (whole && c + kEach <= rows_n) {
                __builtin_nontemporal_store(*reinterpret_cast<const v4u*>(from), reinterpret_cast<v4u*>(to));
            } else {
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    if (c + e >= rows_n) break;
                    if constexpr (kElem == 4) reinterpret_cast<uint32_t*>(to)[e] = reinterpret_cast<const uint32_t*>(from)[e];
                    else reinterpret_cast<uint16_t*>(to)[e] = reinterpret_cast<const uint16_t*>(from)[e];
                }
            }
        }
        rows_done();
    }
}

template <int FM, int FN>
hipError_t launch(const MxGemmArgs& g, hipStream_t stream) {
    using T = Tile<FM, FN>;
    const dim3 grid((unsigned)(ceil_div(g.a.rows, T::BM) * ceil_div(g.b.rows, T::BN)));
    if (g.out_dtype == I8MP_DTYPE_F32) hipLaunchKernelGGL((mx4_gemm_kernel<FM, FN, I8MP_DTYPE_F32>), grid, dim3(256), 0, stream, g);
    else if (g.out_dtype == I8MP_DTYPE_F16) hipLaunchKernelGGL((mx4_gemm_kernel<FM, FN, I8MP_DTYPE_F16>), grid, dim3(256), 0, stream, g);
    else hipLaunchKernelGGL((mx4_gemm_kernel<FM, FN, I8MP_DTYPE_BF16>), grid, dim3(256), 0, stream, g);
    return hipGetLastError();
}

}  // namespace

size_t mx4_gemm_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx4_gemm(const MxGemmArgs& g, hipStream_t stream) {
    const auto tiles = [&](int64_t bm, int64_t bn) { return ceil_div(g.a.rows, bm) * ceil_div(g.b.rows, bn); };
    if (tiles(256, 256) >= 200) return launch<4, 4>(g, stream);
    if (tiles(128, 128) >= 200) return launch<2, 2>(g, stream);
    return launch<1, 1>(g, stream);
}

}  // namespace i8mp
