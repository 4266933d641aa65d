// Product of a few rows with a microscaled 4-bit matrix: the linear of single tokens.
//   out[i, j] = sum_k x[i, k] w[j, k] + bias[j],   x [m x k], m <= 16
// w is read once from memory, straight into the matrix instructions' registers; that
// stream bounds the call.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: a lane holds 32 codes (16 bytes) of one row and their
// scale; lane l has row l % 16 and, of the eight blocks of a stretch of 256 elements, blocks
// 2 (l / 16) and the next, one a step.  w's rows are the first operand: a load of 64 lanes
// covers whole lines of 16 rows as they lie, and a lane's two scales are one 16-bit load.
// The scales of a workgroup's rows come to LDS whole: taken by stretches, 8 bytes of a
// row at a time, they cost 13824 x 5120 1.3 us of 12.5 and 22016 x 8192 7 of 30.
//
// A workgroup of 8 waves has `rows` rows of w (up to 16 R); the waves take stretches in
// turn and meet in LDS at the end, in the order of the waves.  Rows are dealt out so that
// every CU gets as many workgroups of equal work.  Lanes whose row is not there take the
// last row that is: their sums are not stored.
//
// Up to four rows of 16-bit x, of any alignment, are quantized here (kIn), once a workgroup into LDS, while
// the first weights are on their way: a thread's 32 elements are one block.  That saves a
// launch; with more rows every workgroup would read and convert too much of x.
//
// Measured (us of the kernel), weights from memory, 20 matrices in turn: 13824 x 5120 by one row 10.6 (3.6 TB/s of codes and
// scales), by 16 rows quantized before 12.5; 22016 x 8192 22.2 (4.3 TB/s) and 26.  The same 13824 x 5120 again and again
// stays in the last-level cache: 8.4 by one row.
#include "common.h"
#include "mx4.h"
#include "mx4_util.h"

namespace i8mp {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kStretch = 256;            // elements
constexpr int kAhead = 2;                // stretches a wave has on their way

__device__ inline v4i load16(__amdgpu_buffer_rsrc_t src, int offset) {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(src, offset, 0, 0));
}

// bytes of LDS that m rows of quantized x take: codes and scales
__host__ __device__ inline int x_bytes(int64_t m, int64_t k) {
    const int blocks = (int)((k + kStretch - 1) / kStretch) * (kStretch / kMxBlock);
    return (int)m * blocks * 17;
}

// and the scales of `rows` rows of w
__host__ __device__ inline int w_bytes(int64_t rows, int64_t k) {
    return (int)((rows * ((k + kStretch - 1) / kStretch) * (kStretch / kMxBlock) + 15) / 16 * 16);
}

typedef v4u v4u_any __attribute__((aligned(2)));   // at any element's address

// block `id` of x's m rows of `blocks`
__device__ inline void load_x(const MxGemmArgs& g, int blocks, int id, v4u (&v)[4]) {
    const int row = id / blocks, block = id - row * blocks, left = (int)g.a.k - block * kMxBlock;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = v4u{0, 0, 0, 0};
    if (row >= (int)g.a.rows || left <= 0) return;
    const half_bits* p = g.x + row * g.ldx + block * kMxBlock;
    if (left >= kMxBlock) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = reinterpret_cast<const v4u_any*>(p)[e];
    } else {
#pragma unroll
        for (int e = 0; e < kMxBlock; ++e)
            if (e < left) v[e >> 3][e >> 1 & 3] |= (uint32_t)p[e] << (16 * (e & 1));
    }
}
template <bool kBf16>
__device__ inline void quantize_x(const v4u (&v)[4], int id, int all, uint8_t* lds) {
    us2 top = mags(v[0][0]);
#pragma unroll
    for (int e = 1; e < 16; ++e) top = __builtin_elementwise_max(top, mags(v[e >> 2][e & 3]));
    const uint32_t byte = scale_byte<kBf16>(top.x > top.y ? top.x : top.y);
    const float scale = scale_value(byte);
    v4u codes;
#pragma unroll
    for (int e = 0; e < 4; ++e) codes[e] = byte == 255u ? 0u : encode8<kBf16>(v[e][0], v[e][1], v[e][2], v[e][3], scale);
    *reinterpret_cast<v4u*>(lds + id * 16) = codes;
    lds[all * 16 + id] = (uint8_t)byte;
}

// R tiles of 16 rows of w.  kIn: x is quantized (0), fp16 (1) or bfloat16 (2).
template <int R, int kIn, int kType>
__global__ __launch_bounds__(kThreads, 4) void mx4_decode_kernel(MxGemmArgs g, int rows_each) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];   // w's scales, quantized x; later the waves' sums
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int kp = (int)g.a.kp(), stretches = (kp + kStretch - 1) / kStretch, m = (int)g.a.rows;
    const int n0 = (int)blockIdx.x * rows_each, all = (int)g.b.rows;
    const int rows = all - n0 < rows_each ? all - n0 : rows_each;
    const int ldw = (int)g.b.ldc, lsw = (int)g.b.lds, ldx = (int)g.a.ldc, lsx = (int)g.a.lds;
    const __amdgpu_buffer_rsrc_t cw = range_of(g.b.codes + (int64_t)n0 * ldw, kp > 0 ? (rows - 1) * ldw + kp / 2 : 0);
    const __amdgpu_buffer_rsrc_t scales = range_of(g.b.scales + (int64_t)n0 * lsw, kp > 0 ? (rows - 1) * lsw + kp / kMxBlock : 0);
    const __amdgpu_buffer_rsrc_t cx = range_of(g.a.codes, kIn || kp == 0 ? 0 : (m - 1) * ldx + kp / 2);
    const __amdgpu_buffer_rsrc_t sx = range_of(g.a.scales, kIn || kp == 0 ? 0 : (m - 1) * lsx + kp / kMxBlock);
    const int row_scales = stretches * (kStretch / kMxBlock), x_at = w_bytes(rows, kp);
    int ow[R], os[R];   // a lane's places in a first stretch
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = 16 * r + l16 < rows ? 16 * r + l16 : rows - 1;
        ow[r] = row * ldw + quad * 32;
        os[r] = row * row_scales + quad * 2;
    }
    const int x_row = l16 < m ? l16 : m - 1;
    const int ox = kIn ? x_at + (x_row * row_scales + quad * 2) * 16 : x_row * ldx + quad * 32;
    const int oy = kIn ? x_at + m * row_scales * 16 + x_row * row_scales + quad * 2 : x_row * lsx + quad * 2;
    struct Stretch {
        v4i w[R][2], x[2];
        int sx;
    };
    auto fetch = [&](Stretch& b, int t) {
        // the last one may end after 128 elements; those past it are out of range
        const int past = t < stretches && t * kStretch + quad * 64 < kp ? 0 : kOut, at = past ? 0 : t;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            b.w[r][0] = load16(cw, (ow[r] + at * 128) | past);
            b.w[r][1] = load16(cw, (ow[r] + at * 128 + 16) | past);
        }
        if constexpr (kIn == 0) {
            b.x[0] = load16(cx, (ox + at * 128) | past);
            b.x[1] = load16(cx, (ox + at * 128 + 16) | past);
            b.sx = __builtin_amdgcn_raw_buffer_load_b16(sx, (oy + at * 8) | past, 0, 0);
        }
    };
    v4f acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = v4f{};
    auto multiply = [&](Stretch& b, int t) {
        if (t >= stretches) return;
        if constexpr (kIn != 0) {
            b.x[0] = *reinterpret_cast<const v4i*>(lds + ox + t * 128);
            b.x[1] = *reinterpret_cast<const v4i*>(lds + ox + t * 128 + 16);
            b.sx = *reinterpret_cast<const uint16_t*>(lds + oy + t * 8);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int s = *reinterpret_cast<const uint16_t*>(lds + os[r] + t * 8);
            acc[r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b.w[r][0]), operand(b.x[0]), acc[r], 4, 4, 0, s, 0, b.sx);
            acc[r] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b.w[r][1]), operand(b.x[1]), acc[r], 4, 4, 1, s, 1, b.sx);
        }
    };
    Stretch b[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(b[i], wave + i * kWaves);
    const int x_blocks = m * row_scales, words = rows * (row_scales / 4);
    v4u v[4];
    if constexpr (kIn != 0) load_x(g, row_scales, threadIdx.x, v);
    // w's scales, whole rows; past a row's end zeros
    constexpr int kWords = 4;   // a thread's at a time
    for (int base = threadIdx.x; base < words; base += kWords * kThreads) {
        uint32_t word[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int id = base + i * kThreads, row = id / (row_scales / 4), at = (id - row * (row_scales / 4)) * 4;
            word[i] = __builtin_amdgcn_raw_buffer_load_b32(scales, id < words && at < kp / kMxBlock ? row * lsw + at : kOut, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            if (base + i * kThreads < words) reinterpret_cast<uint32_t*>(lds)[base + i * kThreads] = word[i];
    }
    if constexpr (kIn != 0) {
        for (int id = threadIdx.x; id < x_blocks; id += kThreads) {
            if (id >= kThreads) load_x(g, row_scales, id, v);
            quantize_x<kIn == 2>(v, id, x_blocks, lds + x_at);
        }
    }
    __syncthreads();
    for (int t = wave; t < stretches; t += kAhead * kWaves) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            multiply(b[i], t + i * kWaves);
            fetch(b[i], t + (i + kAhead) * kWaves);
        }
    }
    __syncthreads();   // scales and x are done with
    v4f* const sums = reinterpret_cast<v4f*>(lds);
#pragma unroll
    for (int r = 0; r < R; ++r) sums[(wave * R + r) * 64 + lane] = acc[r];
    __syncthreads();
    for (int u = threadIdx.x; u < R * 64; u += kThreads) {
        v4f v = sums[u];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += sums[w * R * 64 + u];
        const int i = u & 15, j = 16 * (u >> 6) + 4 * (u >> 4 & 3);
        if (i >= m) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (j + e >= rows) break;
            const float x = g.bias ? v[e] + widen(g.bias, (int64_t)n0 + j + e, kType) : v[e];
            const int64_t at = (int64_t)i * g.ldout + n0 + j + e;
            if constexpr (kType == I8MP_DTYPE_F32) static_cast<float*>(g.out)[at] = x;
            else static_cast<half_bits*>(g.out)[at] = (half_bits)narrow2<kType>(x, 0.0f);
        }
    }
}

template <int R, int kIn>
hipError_t launch(const MxGemmArgs& g, int rows, hipStream_t stream) {
    const dim3 grid((unsigned)ceil_div(g.b.rows, rows)), block(kThreads);
    const int sums = kWaves * R * 64 * 16, held = w_bytes(rows, g.a.k) + (kIn ? x_bytes(g.a.rows, g.a.k) : 0);
    const int bytes = held > sums ? held : sums;
    if constexpr (kIn == 0)
        if (g.out_dtype == I8MP_DTYPE_F32) hipLaunchKernelGGL((mx4_decode_kernel<R, kIn, I8MP_DTYPE_F32>), grid, block, bytes, stream, g, rows);
    if constexpr (kIn != 2)
        if (g.out_dtype == I8MP_DTYPE_F16) hipLaunchKernelGGL((mx4_decode_kernel<R, kIn, I8MP_DTYPE_F16>), grid, block, bytes, stream, g, rows);
    if constexpr (kIn != 1)
        if (g.out_dtype == I8MP_DTYPE_BF16) hipLaunchKernelGGL((mx4_decode_kernel<R, kIn, I8MP_DTYPE_BF16>), grid, block, bytes, stream, g, rows);
    return hipGetLastError();
}
constexpr int kMaxLds = 64 << 10;

// rows of w that a workgroup can have beside `x` bytes of LDS
int64_t rows_fit(int64_t k, int x) { return (kMaxLds - x - 16) / (round_up(k, kStretch) / kMxBlock + 1); }

// Quantizing x: two workgroups a CU, up to 32 rows each.  x quantized before: one of up to 64 rows, since each reads all
// of x.  us of 16 rows by 5120 x 13824 and 13824 x 5120: 17.2 and 15.0 with two, 15.5 and 14.1 with one; one row that
// is quantized here: 11.1 and 11.2 with two, 12.1 and 12.2 with one.
template <int kIn>
hipError_t launch_rows(const MxGemmArgs& g, hipStream_t stream) {
    constexpr int kGroups = kIn ? 512 : 256;
    const int64_t fit = rows_fit(g.a.k, kIn ? x_bytes(g.a.rows, g.a.k) : 0), most = fit < (kIn ? 32 : 64) ? fit : kIn ? 32 : 64;
    const int64_t rounds = ceil_div(g.b.rows, kGroups * most);
    const int64_t each = ceil_div(g.b.rows, kGroups * rounds), rows = each < 4 && most >= 4 ? 4 : each;
    if (rows <= 16) return launch<1, kIn>(g, (int)rows, stream);
    if constexpr (kIn == 0)
        if (rows > 32) return launch<4, kIn>(g, (int)rows, stream);
    return launch<2, kIn>(g, (int)rows, stream);
}

}  // namespace

bool mx4_decode_fits(int64_t m, int64_t k) { return m <= kMxDecodeRows && rows_fit(k, 0) >= 4; }

bool mx4_decode_quantizes(int64_t m, int64_t k) { return m <= 4 && k > 0 && k <= (1 << 20) && rows_fit(k, x_bytes(m, k)) >= 4; }

hipError_t launch_mx4_decode(const MxGemmArgs& g, hipStream_t stream) {
    if (g.x) return g.out_dtype == I8MP_DTYPE_BF16 ? launch_rows<2>(g, stream) : launch_rows<1>(g, stream);
    return launch_rows<0>(g, stream);
}

}  // namespace i8mp
